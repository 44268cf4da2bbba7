"""Thin ctypes binding of libtile_gemm.so (include/tile_gemm.h).

Argument marshalling only: torch supplies device memory and the current
stream; every step of the product runs in the library's HIP kernels. There is
no fallback: if the library is missing, loading it raises.
"""

from __future__ import annotations

import ctypes
import enum
import os
import struct

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libtile_gemm.so")
_lib = None


class Status(enum.IntEnum):
    OK = 0
    ERR_NULL_ARG = 1
    ERR_BAD_SHAPE = 2
    ERR_BAD_STRIDE = 3
    ERR_MISALIGNED = 4
    ERR_ALIAS = 5
    ERR_DTYPE = 6
    ERR_DEVICE = 7
    ERR_HIP = 8
    ERR_EPILOGUE = 9
    ERR_WORKSPACE = 10


class Dtype(enum.IntEnum):
    BF16_TO_F32 = 0
    BF16_TO_BF16 = 1


class Act(enum.IntEnum):
    NONE = 0
    RELU = 1
    SIGMOID = 2
    TANH = 3
    SILU = 4
    SWIGLU = 5


class Gate(enum.IntEnum):
    """Activation of a gated block's gate half (tile_gemm_gate_t)."""
    SILU = 0
    GELU = 1
    GELU_TANH = 2
    RELU = 3
    SIGMOID = 4


class TrainProduct(enum.IntEnum):
    """Products of the gated block and the cross entropy (tile_gemm_plan_train)."""
    LOGITS = 0
    GATED = 1
    GRADIENT = 2


class IndexType(enum.IntEnum):
    I32 = 0
    I64 = 1


class Quant(enum.IntEnum):
    """What shares a scale (tile_gemm_quant_t)."""
    ROWS = 0
    GATED_ROWS = 1
    BLOCKS = 2


class Score(enum.IntEnum):
    """A router's scores (tile_gemm_score_t)."""
    SOFTMAX = 0
    SIGMOID = 1


DEBUG_COUNT_WRITES = 1
DEBUG_COLLIDE = 2


def DEBUG_FORCE_TILE(c: int) -> int:
    return ((c + 1) & 0xFF) << 8


def DEBUG_FORCE_SKINNY(c: int) -> int:
    return ((c + 1) & 0xFF) << 16


def DEBUG_FORCE_GRID(g: int) -> int:
    return (g & 0x7F) << 24


DEBUG_ONE_TILE_PER_WG = 0x7F << 24


def DEBUG_GROUP_M(g: int) -> int:
    return (g & 0x3F) << 2


N_TILE_CONFIGS = 29
N_MX_CONFIGS = 8
MX_E4M3 = 0
MX_E2M1 = 1
N_SKINNY_CONFIGS = 6

VARIANT_NONE, VARIANT_TILE, VARIANT_SKINNY, VARIANT_MX = 0, 1, 2, 3


class Strides(ctypes.Structure):
    _fields_ = [("a_m", ctypes.c_int64), ("a_k", ctypes.c_int64),
                ("b_k", ctypes.c_int64), ("b_n", ctypes.c_int64),
                ("c_m", ctypes.c_int64), ("c_n", ctypes.c_int64)]


class Plan(ctypes.Structure):
    _fields_ = [("variant", ctypes.c_int32), ("config", ctypes.c_int32),
                ("bm", ctypes.c_int32), ("bn", ctypes.c_int32), ("bk", ctypes.c_int32),
                ("threads", ctypes.c_int32), ("lds_bytes", ctypes.c_int32),
                ("tiles_m", ctypes.c_int32), ("tiles_n", ctypes.c_int32),
                ("group_m", ctypes.c_int32), ("xcds", ctypes.c_int32),
                ("k_split", ctypes.c_int32), ("grid", ctypes.c_int64),
                ("tiles", ctypes.c_int64)]

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}


class XentOptions(ctypes.Structure):
    """Options of the cross entropy (tile_gemm_xent_t)."""
    _fields_ = [("ignore_index", ctypes.c_int64), ("label_smoothing", ctypes.c_float),
                ("z_loss", ctypes.c_float), ("piece", ctypes.c_int64), ("target_type", ctypes.c_int32)]


class Fp8Strides(ctypes.Structure):
    """Strides of the E4M3 products (tile_gemm_fp8_strides_t)."""
    _fields_ = [(n, ctypes.c_int64) for n in ("a_stride", "b_stride", "c_stride", "a_scale_stride",
                                              "b_scale_stride", "b_expert_stride", "b_scale_expert_stride")]


# a Fp8Strides for one call, in a third of the time of a ctypes structure
_fp8_strides = struct.Struct("=7q").pack


class RouteOptions(ctypes.Structure):
    """Options of the routing to experts (tile_gemm_route_t)."""
    _fields_ = [("score", ctypes.c_int32), ("logits_type", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("top_groups", ctypes.c_int32), ("group_top", ctypes.c_int32), ("renormalize", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class TileGemmError(RuntimeError):
    def __init__(self, status, detail=""):
        self.status = Status(status)
        self.detail = detail
        super().__init__(f"{self.status.name}: {status_text(status)}"
                         + (f" ({detail})" if detail else ""))


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load libtile_gemm.so once; raise if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise FileNotFoundError(
            f"{_LIB_PATH} is missing: build it with `python -m tile_partitioned_dense_amd.build`"
            " (there is no fallback implementation)")
    lib = ctypes.CDLL(_LIB_PATH)
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    P = ctypes.POINTER
    lib.tile_gemm_create.argtypes = [P(vp), i32]
    lib.tile_gemm_create.restype = i32
    lib.tile_gemm_destroy.argtypes = [vp]
    lib.tile_gemm_destroy.restype = i32
    lib.tile_gemm_run.argtypes = [vp, vp, vp, vp, i64, i64, i64, P(Strides), i32, vp]
    lib.tile_gemm_run.restype = i32
    lib.tile_gemm_run_debug.argtypes = [vp, vp, vp, vp, i64, i64, i64, P(Strides), i32, vp,
                                        vp, i32, vp, i32]
    lib.tile_gemm_run_debug.restype = i32
    lib.tile_gemm_run_epilogue.argtypes = [vp, vp, vp, vp, i64, i64, i64, P(Strides), i32, vp, i32,
                                           vp]
    lib.tile_gemm_run_epilogue.restype = i32
    lib.tile_gemm_check_epilogue.argtypes = [vp, i64, i64, P(Strides), i32, vp, i32]
    lib.tile_gemm_check_epilogue.restype = i32
    lib.tile_gemm_status_str.argtypes = [i32]
    lib.tile_gemm_status_str.restype = ctypes.c_char_p
    lib.tile_gemm_last_error_detail.argtypes = []
    lib.tile_gemm_last_error_detail.restype = ctypes.c_char_p
    lib.tile_gemm_check_args.argtypes = [vp, vp, vp, i64, i64, i64, P(Strides), i32]
    lib.tile_gemm_check_args.restype = i32
    lib.tile_gemm_plan.argtypes = [i64, i64, i64, i32, i32, P(Plan)]
    lib.tile_gemm_plan.restype = i32
    lib.tile_gemm_plan_mx.argtypes = [i64, i64, i64, i32, i32, P(Plan)]
    lib.tile_gemm_plan_mx.restype = i32
    lib.tile_gemm_run_mx.argtypes = [vp, vp, vp, vp, i64, i64, i64, P(Strides), vp, vp, i64, i32,
                                     i32, vp, i32, vp]
    lib.tile_gemm_run_mx.restype = i32
    lib.tile_gemm_run_mx_debug.argtypes = [vp, vp, vp, vp, i64, i64, i64, P(Strides), vp, vp, i64,
                                           i32, i32, vp, i32, vp, vp, i32]
    lib.tile_gemm_run_mx_debug.restype = i32
    lib.tile_gemm_check_mx.argtypes = [vp, vp, vp, i64, i64, i64, P(Strides), vp, vp, i64, i32, i32,
                                       vp, i32]
    lib.tile_gemm_check_mx.restype = i32
    PX = P(XentOptions)
    lib.tile_gemm_run_glu.argtypes = [vp, vp, vp, vp, i64, i64, i64, P(Strides), i32, vp, i32, vp]
    lib.tile_gemm_run_glu_backward.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, P(Strides),
                                               P(Strides), vp, vp, i32, vp, i64, vp]
    lib.tile_gemm_check_glu_backward.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, P(Strides),
                                                 P(Strides), vp, vp, i32, vp, i64]
    lib.tile_gemm_glu_backward_workspace.argtypes = [vp, i64, i64, i64, P(i64)]
    lib.tile_gemm_run_xent.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, P(Strides), PX, vp,
                                       i64, vp]
    lib.tile_gemm_check_xent.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, P(Strides), PX, vp, i64]
    lib.tile_gemm_xent_workspace.argtypes = [vp, i64, i64, i64, PX, P(i64)]
    lib.tile_gemm_run_xent_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64,
                                                P(Strides), P(Strides), PX, vp, i64, vp]
    lib.tile_gemm_check_xent_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, i64, i64, i64,
                                                  P(Strides), P(Strides), PX, vp, i64]
    lib.tile_gemm_xent_backward_workspace.argtypes = [vp, i64, i64, i64, P(Strides), PX, P(i64)]
    lib.tile_gemm_plan_train.argtypes = [i64, i64, i64, i32, i32, P(Plan)]
    for name in ("plan_train", "run_glu", "run_glu_backward", "check_glu_backward", "glu_backward_workspace",
                 "run_xent", "check_xent", "xent_workspace", "run_xent_backward",
                 "check_xent_backward", "xent_backward_workspace"):
        getattr(lib, "tile_gemm_" + name).restype = i32
    PF, PR = P(Fp8Strides), P(RouteOptions)
    lib.tile_gemm_check_fp8.argtypes = [vp, vp, vp, i64, i64, i64, PF, vp, vp, i32, vp, i32]
    # (the products take their strides as bytes, too)
    lib.tile_gemm_run_fp8.argtypes = [vp, *(vp if t is PF else t for t in lib.tile_gemm_check_fp8.argtypes), vp]
    lib.tile_gemm_check_fp8_experts.argtypes = [vp, vp, vp, i64, i64, i64, i64, vp, PF, vp, vp, i32]
    lib.tile_gemm_run_fp8_experts.argtypes = [
        vp, *(vp if t is PF else t for t in lib.tile_gemm_check_fp8_experts.argtypes), vp]
    lib.tile_gemm_check_quantize.argtypes = [vp, vp, vp, i64, i64, i64, i64, i64, i32, i32, vp, i64]
    lib.tile_gemm_run_quantize.argtypes = [vp, *lib.tile_gemm_check_quantize.argtypes, vp]
    lib.tile_gemm_check_route.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, PR]
    lib.tile_gemm_run_route.argtypes = [vp, *lib.tile_gemm_check_route.argtypes, vp]
    lib.tile_gemm_check_route_backward.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, i64, PR]
    lib.tile_gemm_run_route_backward.argtypes = [vp, *lib.tile_gemm_check_route_backward.argtypes, vp]
    lib.tile_gemm_check_place.argtypes = [vp, i64, i64, i64, i64, vp, vp, vp, vp, i64]
    lib.tile_gemm_run_place.argtypes = [vp, *lib.tile_gemm_check_place.argtypes, vp]
    lib.tile_gemm_place_workspace.argtypes = [i64, i64, i64, P(i64)]
    lib.tile_gemm_check_combine.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, i64, i64, i32]
    lib.tile_gemm_run_combine.argtypes = [vp, *lib.tile_gemm_check_combine.argtypes, vp]
    lib.tile_gemm_plan_fp8.argtypes = [i64, i64, i64, i64, i32, i32, P(Plan)]
    for name in ("fp8", "fp8_experts", "quantize", "route", "route_backward", "place", "combine"):
        getattr(lib, "tile_gemm_run_" + name).restype = i32
        getattr(lib, "tile_gemm_check_" + name).restype = i32
    lib.tile_gemm_place_workspace.restype = i32
    lib.tile_gemm_plan_fp8.restype = i32
    lib.tile_gemm_tile_of.argtypes = [P(Plan), i64, i64, i64, P(i64), P(i64), P(i64), P(i64)]
    lib.tile_gemm_tile_of.restype = i32
    _lib = lib
    return lib


def status_text(s) -> str:
    return load_library().tile_gemm_status_str(int(s)).decode()


tile_gemm_status_str = status_text


def last_error_detail() -> str:
    return load_library().tile_gemm_last_error_detail().decode()


def _raise_if(st):
    if st != Status.OK:
        raise TileGemmError(st, last_error_detail())


# ----------------------------------------------------------------- handles

def tile_gemm_create(device: int = 0):
    """Create a handle for HIP device `device` (must be gfx950)."""
    lib = load_library()
    h = ctypes.c_void_p()
    _raise_if(lib.tile_gemm_create(ctypes.byref(h), int(device)))
    return h


def tile_gemm_destroy(h) -> None:
    _raise_if(load_library().tile_gemm_destroy(h))


# ----------------------------------------------------------------- marshalling

def _is_tensor(x):
    return hasattr(x, "data_ptr") and hasattr(x, "stride")


def _check_devices(named):
    """The library sees raw pointers only, so the binding checks what it cannot:
    every tensor argument lives on the GPU that is current (the device the
    library launches on), all on the same one. A host tensor's pointer handed
    to a kernel would fault the GPU."""
    import torch
    cur = torch.cuda.current_device() if torch.cuda.is_available() else None
    for name, t in named:
        if t is None or not _is_tensor(t):
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} is on {t.device}; every tensor argument must be on the GPU")
        if t.device.index != cur:
            raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{cur}")


def _check_bias(bias, n):
    """A bias tensor must be a contiguous vector of n float32 values (the
    kernels read exactly that many)."""
    import torch
    if bias is None or not _is_tensor(bias):
        return
    if bias.dtype != torch.float32:
        raise TypeError(f"bias must be float32, got {bias.dtype}")
    if bias.dim() != 1 or bias.numel() != n or not bias.is_contiguous():
        raise ValueError(f"bias must be a contiguous vector of {n} values, got shape "
                         f"{tuple(bias.shape)} strides {tuple(bias.stride())}")


def _check_counts(counts, m, n):
    """Write counts: a contiguous 32-bit integer array of at least m*n elements."""
    import torch
    if counts is None or not _is_tensor(counts):
        return
    if counts.dtype not in (torch.int32, getattr(torch, "uint32", torch.int32)):
        raise TypeError(f"counts must be a 32-bit integer tensor, got {counts.dtype}")
    if counts.numel() < m * n or not counts.is_contiguous():
        raise ValueError(f"counts must be contiguous with at least {m * n} elements")


def _c_dtype(C):
    import torch
    if C.dtype == torch.float32:
        return Dtype.BF16_TO_F32
    if C.dtype == torch.bfloat16:
        return Dtype.BF16_TO_BF16
    raise TypeError("C must be float32 or bfloat16")


def _operands(A, B, C, M, N, K, strides, dtype, c_cols_div=1):
    """Pointers, shape, strides and dtype from torch tensors or raw values.
    C has N / c_cols_div columns (2 for SiLU(gate) * up)."""
    if _is_tensor(A) and _is_tensor(B) and _is_tensor(C):
        import torch
        if A.dim() != 2 or B.dim() != 2 or C.dim() != 2:
            raise ValueError("A, B and C must be 2-D")
        if A.dtype != torch.bfloat16 or B.dtype != torch.bfloat16:
            raise TypeError("A and B must be bfloat16")
        M_, K_ = A.shape
        K2, N_ = B.shape
        if K2 != K_ or N_ % c_cols_div or tuple(C.shape) != (M_, N_ // c_cols_div):
            raise ValueError(f"shapes do not chain: A{tuple(A.shape)} B{tuple(B.shape)} "
                             f"C{tuple(C.shape)}")
        cdt = _c_dtype(C)
        if dtype is None:
            dtype = cdt
        elif int(dtype) != cdt:
            raise TypeError(f"dtype {Dtype(int(dtype)).name} does not match C's {C.dtype}")
        s = Strides(A.stride(0), A.stride(1), B.stride(0), B.stride(1), C.stride(0), C.stride(1))
        return (A.data_ptr(), B.data_ptr(), C.data_ptr(), M_, N_, K_, s, int(dtype))
    if any(_is_tensor(x) for x in (A, B, C)):
        raise TypeError("A, B and C must be all torch tensors or all raw pointers")
    if None in (M, N, K, strides, dtype):
        raise ValueError("raw pointers need M, N, K, strides and dtype")
    s = strides if isinstance(strides, Strides) else Strides(*strides)
    return (A, B, C, int(M), int(N), int(K), s, int(dtype))


def _stream_ptr(stream, C):
    if stream is None:
        if _is_tensor(C) and C.is_cuda:
            import torch
            return torch.cuda.current_stream(C.device).cuda_stream
        return None
    if hasattr(stream, "cuda_stream"):
        return stream.cuda_stream
    return int(stream)


def tile_gemm_run(h, A, B, C, M=None, N=None, K=None, strides=None, dtype=None, stream=None,
                  check: bool = True):
    """Enqueue C := A.B. With torch tensors the shape, strides, output dtype and
    (unless given) the current stream are taken from them. Returns the status;
    raises TileGemmError on a non-OK status when `check` is true."""
    a, b, c, M_, N_, K_, s, dt = _operands(A, B, C, M, N, K, strides, dtype)
    _check_devices((("A", A), ("B", B), ("C", C)))
    st = load_library().tile_gemm_run(h, a, b, c, M_, N_, K_, ctypes.byref(s), dt,
                                      _stream_ptr(stream, C))
    if check:
        _raise_if(st)
    return Status(st)


def tile_gemm_run_epilogue(h, A, B, C, bias=None, act=Act.NONE, M=None, N=None, K=None,
                           strides=None, dtype=None, stream=None, check: bool = True):
    """Enqueue C := act(A.B + bias) (bias: N fp32 values on the device, or None).
    With act=Act.SWIGLU, C is M x N/2: silu of B's first N/2 columns' results
    times its last N/2."""
    div = 2 if int(act) == Act.SWIGLU else 1
    a, b, c, M_, N_, K_, s, dt = _operands(A, B, C, M, N, K, strides, dtype, div)
    _check_bias(bias, N_)
    _check_devices((("A", A), ("B", B), ("C", C), ("bias", bias)))
    bp = bias.data_ptr() if _is_tensor(bias) else bias
    st = load_library().tile_gemm_run_epilogue(h, a, b, c, M_, N_, K_, ctypes.byref(s), dt, bp,
                                               int(act), _stream_ptr(stream, C))
    if check:
        _raise_if(st)
    return Status(st)


def tile_gemm_run_debug(h, A, B, C, counts=None, flags=0, M=None, N=None, K=None, strides=None,
                        dtype=None, stream=None, check: bool = True, bias=None, act=Act.NONE):
    """tile_gemm_run (or, with bias/act, tile_gemm_run_epilogue) with test
    instrumentation (write counts, collision, forced configuration or grid)."""
    div = 2 if int(act) == Act.SWIGLU else 1
    a, b, c, M_, N_, K_, s, dt = _operands(A, B, C, M, N, K, strides, dtype, div)
    _check_bias(bias, N_)
    _check_counts(counts, M_, N_ // div)
    _check_devices((("A", A), ("B", B), ("C", C), ("bias", bias), ("counts", counts)))
    cnt = counts.data_ptr() if _is_tensor(counts) else counts
    bp = bias.data_ptr() if _is_tensor(bias) else bias
    st = load_library().tile_gemm_run_debug(h, a, b, c, M_, N_, K_, ctypes.byref(s), dt,
                                            _stream_ptr(stream, C), cnt, int(flags), bp,
                                            int(act))
    if check:
        _raise_if(st)
    return Status(st)


def _mx_operands(A, Bt, C, a_scale, b_scale, fmt=MX_E4M3):
    """Pointers, shape and strides of an MX call from torch tensors: A (M x K)
    and Bt (N x K) uint8 E4M3 codes (E2M1: M x K/2 and N x K/2 packed bytes),
    scales uint8 (M x ls) and (N x ls)."""
    import torch
    for name, t in (("A", A), ("Bt", Bt), ("a_scale", a_scale), ("b_scale", b_scale)):
        if t.dtype != torch.uint8 or t.dim() != 2:
            raise TypeError(f"{name} must be a 2-D uint8 tensor")
    M, K = A.shape
    N, K2 = Bt.shape
    if fmt == MX_E2M1:
        K, K2 = 2 * K, 2 * K2
    if K2 != K or tuple(C.shape) != (M, N):
        raise ValueError(f"shapes do not chain: A{tuple(A.shape)} Bt{tuple(Bt.shape)} C{tuple(C.shape)}")
    if a_scale.shape[0] != M or b_scale.shape[0] != N or a_scale.stride(1) != 1 \
            or b_scale.stride(1) != 1:
        raise ValueError("scales: M and N rows with unit column stride")
    # One row stride serves both scale arrays. The stride of a single-row
    # array is never used (and torch may report any value for it), so it takes
    # the other array's; two single rows use their row length.
    if M > 1 and N > 1 and a_scale.stride(0) != b_scale.stride(0):
        raise ValueError("scales: A's and B's scale rows must have one common stride")
    ls = a_scale.stride(0) if M > 1 else (b_scale.stride(0) if N > 1 else a_scale.shape[1])
    dtype = _c_dtype(C)
    s = Strides(A.stride(0), A.stride(1), Bt.stride(1), Bt.stride(0), C.stride(0), C.stride(1))
    return M, N, K, s, ls, int(dtype)


def tile_gemm_run_mx(h, A, Bt, C, a_scale, b_scale, bias=None, act=Act.NONE, stream=None,
                     counts=None, flags=0, check: bool = True, fmt=MX_E4M3):
    """Enqueue the MX product C := act((sa * A) . (sb * Bt)^T + bias) (torch tensors)."""
    M, N, K, s, ls, dt = _mx_operands(A, Bt, C, a_scale, b_scale, fmt)
    _check_bias(bias, N)
    _check_counts(counts, M, N)
    _check_devices((("A", A), ("Bt", Bt), ("C", C), ("a_scale", a_scale), ("b_scale", b_scale),
                    ("bias", bias), ("counts", counts)))
    bp = bias.data_ptr() if _is_tensor(bias) else bias
    lib = load_library()
    args = (h, A.data_ptr(), Bt.data_ptr(), C.data_ptr(), M, N, K, ctypes.byref(s),
            a_scale.data_ptr(), b_scale.data_ptr(), ls, int(fmt), dt, bp, int(act),
            _stream_ptr(stream, C))
    if flags or counts is not None:
        cnt = counts.data_ptr() if _is_tensor(counts) else counts
        st = lib.tile_gemm_run_mx_debug(*args, cnt, int(flags))
    else:
        st = lib.tile_gemm_run_mx(*args)
    if check:
        _raise_if(st)
    return Status(st)


# ------------------------------------------------ gated block, cross entropy
# A call on few rows takes the GPU a few microseconds, so these bindings keep
# what they do for each call short: one comparison per argument, and the long
# form of a check only to word its error.

def _matrix(name, t, rows, cols):
    """Checks a 2-D bf16 tensor (rows, cols None: any); its shape."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
    s = t.shape
    if len(s) != 2 or (rows is not None and s[0] != rows) or (cols is not None and s[1] != cols):
        raise ValueError(f"{name} must have shape ({'any' if rows is None else rows}, "
                         f"{'any' if cols is None else cols}), got {tuple(s)}")
    return s


def _vector(name, t, n, dtypes):
    """Checks a contiguous vector of n values."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {[str(d) for d in dtypes]}, got {t.dtype}")
    s = t.shape
    if len(s) != 1 or s[0] != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of {n} values, got shape "
                         f"{tuple(s)} strides {tuple(t.stride())}")


def _current_device(names, tensors):
    """The current device, on which every tensor has to be."""
    import torch
    # (the first tensor on a GPU means that there is one; asking torch whether
    # there is costs as much as a launch's share of the call)
    cur = torch._C._cuda_getDevice() if tensors[0].is_cuda else None
    for t in tensors:
        if t is not None and t.get_device() != cur:
            _check_devices(zip(names, tensors))
    return cur


def _col_major_strides(b):
    """(b_k, b_n) of a column-major K x N operand; an axis of one element has
    no stride of its own (torch may report any value for it)."""
    b_k, b_n = b.stride()
    K, N = b.shape
    if K == 1:
        b_k = 1
    if N <= 1:
        b_n = max(b_n, K)
    return b_k, b_n


def _row_major_strides(t):
    """(row, column) strides of a row-major matrix; see _col_major_strides."""
    row, col = t.stride()
    return row, (1 if col != 1 and t.shape[1] <= 1 else col)


def _launch_stream(stream, device):
    """The raw stream of a call on the current device, and the stream a
    workspace allocated for it has to be handed over to (None: the current)."""
    import torch
    cur = torch._C._cuda_getCurrentRawStream(device)
    if stream is None:
        return cur, None
    raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if raw == cur:
        return cur, None
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(raw, device=torch.device("cuda", device))
    return raw, stream


def _own_workspace(nbytes, near, device, other):
    """A workspace for one call beside the tensor `near`; torch keeps its
    memory until the stream has passed the call."""
    import torch
    ws = near.new_empty(nbytes or 1, dtype=torch.uint8)
    if other is not None:
        ws.record_stream(other)
        # the block may have been freed on the current stream while work
        # queued there still uses it
        other.wait_stream(torch.cuda.current_stream(device))
    return ws


def _workspace_bytes(ws):
    if not _is_tensor(ws) or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor")
    return ws.numel() * ws.element_size()


def _result(st, check):
    if st:
        if check:
            _raise_if(st)
        return Status(st)
    return Status.OK


def tile_gemm_run_glu(h, A, B, C, gate=Gate.SILU, bias=None, stream=None, check: bool = True):
    """Enqueue the gated block C := act(A.B_gate + b_gate) * (A.B_up + b_up)
    (torch tensors; B is K x N with the N/2 gate columns first, either layout;
    C is M x N/2, float32 or bfloat16)."""
    M, K = _matrix("A", A, None, None)
    N = _matrix("B", B, K, None)[1]
    if not _is_tensor(C) or C.dim() != 2 or N % 2 or tuple(C.shape) != (M, N // 2):
        raise ValueError(f"C must be a tensor of shape {(M, N // 2)} for B{tuple(B.shape)}")
    dt = _c_dtype(C)
    if bias is not None:
        _check_bias(bias, N)
    dev = _current_device(("A", "B", "C", "bias"), (A, B, C, bias if _is_tensor(bias) else None))
    s = Strides(*_row_major_strides(A), *B.stride(), *C.stride())
    if M == 1:  # the stride from a single row to the next is never used
        s.a_m, s.c_m = (K + 7) // 8 * 8, (N // 2 + 7) // 8 * 8
    raw, _ = _launch_stream(stream, dev)
    st = load_library().tile_gemm_run_glu(h, A.data_ptr(), B.data_ptr(), C.data_ptr(), M, N, K,
                                          ctypes.byref(s), dt,
                                          bias.data_ptr() if _is_tensor(bias) else bias, gate, raw)
    return _result(st, check)


def tile_gemm_glu_backward_workspace(h, M, N, K) -> int:
    """Workspace bytes of tile_gemm_run_glu_backward (h None: an MI355X)."""
    n = ctypes.c_int64()
    _raise_if(load_library().tile_gemm_glu_backward_workspace(h, M, N, K, ctypes.byref(n)))
    return n.value


def tile_gemm_run_glu_backward(h, A, B, dC, dA=None, dB=None, gate=Gate.SILU, bias=None, dbias=None,
                               workspace=None, stream=None, check: bool = True):
    """Enqueue the backward pass of the gated block (torch tensors): dA (M x K),
    dB (K x N, column-major like B) and dbias (N float32) from dC (M x N/2);
    any of the three may be left out. Without `workspace` one is allocated for
    the call."""
    import torch
    M, K = _matrix("A", A, None, None)
    N = _matrix("B", B, K, None)[1]
    _matrix("dC", dC, M, N // 2)
    s = Strides(*_row_major_strides(A), *_col_major_strides(B), 0, 0)
    g = Strides(0, 1, 1, 0, *_row_major_strides(dC))
    p_dA = p_dB = p_bias = p_dbias = None
    if dA is not None:
        _matrix("dA", dA, M, K)
        g.a_m, g.a_k = _row_major_strides(dA)
        p_dA = dA.data_ptr()
    if dB is not None:
        _matrix("dB", dB, K, N)
        g.b_k, g.b_n = _col_major_strides(dB)
        p_dB = dB.data_ptr()
    if bias is not None:
        _vector("bias", bias, N, (torch.float32,))
        p_bias = bias.data_ptr()
    if dbias is not None:
        _vector("dbias", dbias, N, (torch.float32,))
        p_dbias = dbias.data_ptr()
    dev = _current_device(("A", "B", "dC", "dA", "dB", "bias", "dbias", "workspace"),
                          (A, B, dC, dA, dB, bias, dbias, workspace))
    raw, other = _launch_stream(stream, dev)
    if workspace is None:
        nbytes = tile_gemm_glu_backward_workspace(h, M, N, K)
        workspace = _own_workspace(nbytes, A, dev, other)
    else:
        nbytes = _workspace_bytes(workspace)
    st = load_library().tile_gemm_run_glu_backward(
        h, A.data_ptr(), B.data_ptr(), dC.data_ptr(), p_dA, p_dB, M, N, K, ctypes.byref(s),
        ctypes.byref(g), p_bias, p_dbias, gate, workspace.data_ptr(), nbytes, raw)
    return _result(st, check)


def _xent_operands(A, B, target, ignore_index, label_smoothing, z_loss, piece):
    import torch
    M, K = _matrix("A", A, None, None)
    N = _matrix("B", B, K, None)[1]
    _vector("target", target, M, (torch.int64, torch.int32))
    s = Strides(*_row_major_strides(A), *_col_major_strides(B), 0, 0)
    o = XentOptions(ignore_index, label_smoothing, z_loss, piece, target.dtype is torch.int64)
    return M, N, K, s, o


def tile_gemm_xent_workspace(h, M, N, K, label_smoothing=0.0) -> int:
    """Workspace bytes of tile_gemm_run_xent (h None: an MI355X)."""
    n = ctypes.c_int64()
    o = XentOptions(0, label_smoothing, 0.0, 0, 0)
    _raise_if(load_library().tile_gemm_xent_workspace(h, M, N, K, ctypes.byref(o), ctypes.byref(n)))
    return n.value


def tile_gemm_run_xent(h, A, B, target, loss=None, lse=None, ignore_index=-100, label_smoothing=0.0,
                       z_loss=0.0, workspace=None, stream=None, check: bool = True):
    """Enqueue the per-row cross entropy of the projection A.B onto B's N
    columns (torch tensors; B K x N column-major): loss and lse, M float32
    values each, without storing the logits."""
    import torch
    M, N, K, s, o = _xent_operands(A, B, target, ignore_index, label_smoothing, z_loss, 0)
    p_loss = p_lse = None
    if loss is not None:
        _vector("loss", loss, M, (torch.float32,))
        p_loss = loss.data_ptr()
    if lse is not None:
        _vector("lse", lse, M, (torch.float32,))
        p_lse = lse.data_ptr()
    dev = _current_device(("A", "B", "target", "loss", "lse", "workspace"),
                          (A, B, target, loss, lse, workspace))
    lib = load_library()
    raw, other = _launch_stream(stream, dev)
    if workspace is None:
        n = ctypes.c_int64()
        _raise_if(lib.tile_gemm_xent_workspace(h, M, N, K, ctypes.byref(o), ctypes.byref(n)))
        nbytes = n.value
        workspace = _own_workspace(nbytes, A, dev, other)
    else:
        nbytes = _workspace_bytes(workspace)
    st = lib.tile_gemm_run_xent(h, A.data_ptr(), B.data_ptr(), target.data_ptr(), p_loss, p_lse,
                                           M, N, K, ctypes.byref(s), ctypes.byref(o),
                                           workspace.data_ptr(), nbytes, raw)
    return _result(st, check)


def tile_gemm_xent_backward_workspace(h, M, N, K, b_n=None, piece=0) -> int:
    """Workspace bytes of tile_gemm_run_xent_backward (h None: an MI355X) for a
    B whose columns are b_n elements apart (None: K)."""
    n = ctypes.c_int64()
    s = Strides(0, 1, 1, K if b_n is None else b_n, 0, 0)
    o = XentOptions(0, 0.0, 0.0, piece, 0)
    _raise_if(load_library().tile_gemm_xent_backward_workspace(h, M, N, K, ctypes.byref(s), ctypes.byref(o),
                                                               ctypes.byref(n)))
    return n.value


def tile_gemm_run_xent_backward(h, A, B, target, lse, dloss, dA=None, dB=None, ignore_index=-100,
                                label_smoothing=0.0, z_loss=0.0, piece=0, workspace=None, stream=None,
                                check: bool = True):
    """Enqueue the gradients dA (M x K) and dB (K x N, column-major like B) of
    sum(dloss * loss) from tile_gemm_run_xent's lse; either may be left out.
    `piece`: at most this many vocabulary columns at a time (0: chosen)."""
    import torch
    M, N, K, s, o = _xent_operands(A, B, target, ignore_index, label_smoothing, z_loss, piece)
    _vector("lse", lse, M, (torch.float32,))
    _vector("dloss", dloss, M, (torch.float32,))
    g = Strides(0, 1, 1, 0, 0, 1)
    p_dA = p_dB = None
    if dA is not None:
        _matrix("dA", dA, M, K)
        g.a_m, g.a_k = _row_major_strides(dA)
        p_dA = dA.data_ptr()
    if dB is not None:
        _matrix("dB", dB, K, N)
        g.b_k, g.b_n = _col_major_strides(dB)
        p_dB = dB.data_ptr()
    dev = _current_device(("A", "B", "target", "lse", "dloss", "dA", "dB", "workspace"),
                          (A, B, target, lse, dloss, dA, dB, workspace))
    lib = load_library()
    raw, other = _launch_stream(stream, dev)
    if workspace is None:
        n = ctypes.c_int64()
        _raise_if(lib.tile_gemm_xent_backward_workspace(h, M, N, K, ctypes.byref(s), ctypes.byref(o),
                                                        ctypes.byref(n)))
        nbytes = n.value
        workspace = _own_workspace(nbytes, A, dev, other)
    else:
        nbytes = _workspace_bytes(workspace)
    st = lib.tile_gemm_run_xent_backward(
        h, A.data_ptr(), B.data_ptr(), target.data_ptr(), lse.data_ptr(), dloss.data_ptr(), p_dA, p_dB, M,
        N, K, ctypes.byref(s), ctypes.byref(g), ctypes.byref(o), workspace.data_ptr(), nbytes, raw)
    return _result(st, check)


def tile_gemm_plan_train(M, N, K, product, cu_count=256) -> Plan:
    p = Plan()
    _raise_if(load_library().tile_gemm_plan_train(int(M), int(N), int(K), int(product), int(cu_count),
                                                  ctypes.byref(p)))
    return p


def _strides(s):
    return s if s is None or isinstance(s, Strides) else Strides(*s)


def _ref(s):
    return None if s is None else ctypes.byref(s)


def tile_gemm_check_glu_backward(A, B, dC, dA, dB, M, N, K, strides, grad_strides, bias=None, dbias=None,
                                 gate=Gate.SILU, workspace=None, workspace_bytes=0) -> Status:
    """Host-only checks of tile_gemm_run_glu_backward's arguments (pointers are integers)."""
    return Status(load_library().tile_gemm_check_glu_backward(
        A, B, dC, dA, dB, int(M), int(N), int(K), _ref(_strides(strides)), _ref(_strides(grad_strides)), bias,
        dbias, int(gate), workspace, int(workspace_bytes)))


def tile_gemm_check_xent(A, B, target, loss, lse, M, N, K, strides, options, workspace=None,
                         workspace_bytes=0) -> Status:
    """Host-only checks of tile_gemm_run_xent's arguments (pointers are integers)."""
    return Status(load_library().tile_gemm_check_xent(
        A, B, target, loss, lse, int(M), int(N), int(K), _ref(_strides(strides)), _ref(options), workspace,
        int(workspace_bytes)))


def tile_gemm_check_xent_backward(A, B, target, lse, dloss, dA, dB, M, N, K, strides, grad_strides, options,
                                  workspace=None, workspace_bytes=0) -> Status:
    """Host-only checks of tile_gemm_run_xent_backward's arguments (pointers are integers)."""
    return Status(load_library().tile_gemm_check_xent_backward(
        A, B, target, lse, dloss, dA, dB, int(M), int(N), int(K), _ref(_strides(strides)),
        _ref(_strides(grad_strides)), _ref(options), workspace, int(workspace_bytes)))


# ---------------------------- E4M3 products with block scales, routing to experts
# (as above, one look at each tensor's shape and strides; these calls are often
# a microsecond or two of GPU work)

# torch's tensor class, types and current device and stream, looked up once
_torch_names = None


def _names():
    global _torch_names
    import torch
    _torch_names = (torch.Tensor, torch.float8_e4m3fn, torch.uint8, torch.bfloat16, torch.float32, torch.int32,
                    torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream)
    return _torch_names


def _bad(name, t, what):
    raise ValueError(f"{name} must have {what}, got shape {tuple(t.shape)} strides {tuple(t.stride())}")


def _typed(name, t, dtype):
    if not isinstance(t, (_torch_names or _names())[0]):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _e4m3(name, t, dims):
    """Shape and row stride of a tensor of E4M3 codes (float8_e4m3fn, or their bytes as uint8)."""
    tensor, f8, u8 = (_torch_names or _names())[:3]
    if not isinstance(t, tensor):
        raise TypeError(f"{name} must be a torch tensor")
    dtype = t.dtype
    if dtype is not f8 and dtype is not u8:
        raise TypeError(f"{name} must be float8_e4m3fn (or uint8 codes), got {dtype}")
    s, d = t.shape, t.stride()
    if len(s) != dims or (d[-1] != 1 and s[-1] > 1):
        _bad(name, t, f"{dims} dimensions, the last of stride 1")
    return s, d


def _row_scales(name, t, M, kb):
    """The stride between blocks of K of the scales of M rows, (M, blocks of K)
    with rows next to each other."""
    _typed(name, t, (_torch_names or _names())[4])
    s, d = t.shape, t.stride()
    if len(s) != 2 or s[0] != M or s[1] != kb or (d[0] != 1 and M > 1):
        _bad(name, t, f"shape ({M}, {kb}) and a row stride of 1")
    return d[1] if kb > 1 else max(M, 1)


def _block_scales(name, t, lead, nb, kb):
    """The strides of the scales of blocks of 128 x 128, (*lead, blocks of rows, blocks of K)."""
    _typed(name, t, (_torch_names or _names())[4])
    s, d = t.shape, t.stride()
    if s != (*lead, nb, kb) or (d[-1] != 1 and kb > 1):
        _bad(name, t, f"shape {(*lead, nb, kb)} and a last stride of 1")
    return d[-2] if nb > 1 else kb, d[0]


def _rows_of(name, t, M, N):
    """The row stride of an M x N matrix (of a single row, whose stride is any, the
    least that is a whole 16 bytes)."""
    s, d = t.shape, t.stride()
    if s != (M, N) or (d[1] != 1 and N > 1):
        _bad(name, t, f"shape {(M, N)} and a column stride of 1")
    return d[0] if M > 1 else (N + 7) // 8 * 8


def _result_rows(name, t, M, N):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    return (1 if t.dtype is torch.bfloat16 else _c_dtype(t)), _rows_of(name, t, M, N)


def tile_gemm_run_fp8(h, A, Bt, C, a_scale, b_scale, bias=None, act=Act.NONE, stream=None, check: bool = True):
    """Enqueue C := act((a_scale * A) . (b_scale * Bt)^T + bias) with E4M3 A
    (M x K) and Bt (N x K; float8_e4m3fn or uint8 codes) and float32 scales:
    a_scale (M, ceil(K / 128)) with rows next to each other (stride(0) == 1),
    b_scale (ceil(N / 128), ceil(K / 128)), one for each 128 x 128 block."""
    tensor, f8, u8, bf16, f32, _, device, raw_stream = _torch_names or _names()
    # plain tensors of the expected form in one look; anything else step by step
    if (type(A) is tensor and type(Bt) is tensor and type(C) is tensor and type(a_scale) is tensor
            and type(b_scale) is tensor and A.dim() == 2 and Bt.dim() == 2 and C.dim() == 2 and a_scale.dim() == 2
            and b_scale.dim() == 2):
        (M, K), (N, K2), (ta, tb, tc) = A.shape, Bt.shape, (A.dtype, Bt.dtype, C.dtype)
        kb, nb = (K + 127) // 128, (N + 127) // 128
        (a, a1), (b, b1), (c, c1), (x1, x), (y, y1) = (A.stride(), Bt.stride(), C.stride(), a_scale.stride(),
                                                       b_scale.stride())
        plain = (K == K2 and a1 == b1 == c1 == x1 == y1 == 1 and (ta is f8 or ta is u8) and (tb is f8 or tb is u8)
                 and (tc is bf16 or tc is f32) and a_scale.dtype is f32 and b_scale.dtype is f32
                 and C.shape == (M, N) and a_scale.shape == (M, kb) and b_scale.shape == (nb, kb))
    else:
        plain = False
    if plain:
        dt = 1 if tc is bf16 else 0
        s = _fp8_strides(a if M > 1 else K, b if N > 1 else K, c if M > 1 else (N + 7) // 8 * 8,
                         x if kb > 1 else max(M, 1), y if nb > 1 else kb, 0, 0)
    else:
        (M, K), a = _e4m3("A", A, 2)
        (N, K2), b = _e4m3("Bt", Bt, 2)
        if K2 != K:
            raise ValueError(f"shapes do not chain: A{tuple(A.shape)} Bt{tuple(Bt.shape)}")
        dt, ldc = _result_rows("C", C, M, N)
        kb = (K + 127) // 128
        s = _fp8_strides(a[0] if M > 1 else K, b[0] if N > 1 else K, ldc, _row_scales("a_scale", a_scale, M, kb),
                         _block_scales("b_scale", b_scale, (), (N + 127) // 128, kb)[0], 0, 0)
    p_bias = None
    if bias is not None:
        _check_bias(bias, N)
        p_bias = bias.data_ptr() if _is_tensor(bias) else bias
    dev = A.get_device()
    if (p_bias is not None or stream is not None or dev < 0 or Bt.get_device() != dev or C.get_device() != dev
            or a_scale.get_device() != dev or b_scale.get_device() != dev or device() != dev):
        dev = _current_device(("A", "Bt", "C", "a_scale", "b_scale", "bias"),
                              (A, Bt, C, a_scale, b_scale, bias if _is_tensor(bias) else None))
        raw, _ = _launch_stream(stream, dev)
    else:
        raw = raw_stream(dev)
    st = (_lib or load_library()).tile_gemm_run_fp8(h, A.data_ptr(), Bt.data_ptr(), C.data_ptr(), M, N, K,
                                                    s, a_scale.data_ptr(), b_scale.data_ptr(), dt,
                                                    p_bias, act, raw)
    return _result(st, check) if st else Status.OK


def tile_gemm_run_fp8_experts(h, A, Bt, C, a_scale, b_scale, offsets, stream=None, check: bool = True):
    """Enqueue the experts' products: rows [offsets[e], offsets[e + 1]) of C are
    those rows of A times expert e's matrix. Bt (E, N, K), b_scale
    (E, ceil(N / 128), ceil(K / 128)), offsets E + 1 int32 values; A and a_scale
    as for tile_gemm_run_fp8."""
    tensor, f8, u8, bf16, f32, i32, device, raw_stream = _torch_names or _names()
    # (as in tile_gemm_run_fp8)
    if (type(A) is tensor and type(Bt) is tensor and type(C) is tensor and type(a_scale) is tensor
            and type(b_scale) is tensor and A.dim() == 2 and Bt.dim() == 3 and C.dim() == 2 and a_scale.dim() == 2
            and b_scale.dim() == 3):
        (M, K), (E, N, K2), (ta, tb, tc) = A.shape, Bt.shape, (A.dtype, Bt.dtype, C.dtype)
        kb, nb = (K + 127) // 128, (N + 127) // 128
        (a, a1), (be, b, b1), (c, c1), (x1, x), (ye, y, y1) = (A.stride(), Bt.stride(), C.stride(), a_scale.stride(),
                                                               b_scale.stride())
        plain = (K == K2 and a1 == b1 == c1 == x1 == y1 == 1 and (ta is f8 or ta is u8) and (tb is f8 or tb is u8)
                 and (tc is bf16 or tc is f32) and a_scale.dtype is f32 and b_scale.dtype is f32
                 and C.shape == (M, N) and a_scale.shape == (M, kb) and b_scale.shape == (E, nb, kb))
    else:
        plain = False
    if plain:
        dt = 1 if tc is bf16 else 0
        s = _fp8_strides(a if M > 1 else K, b if N > 1 else K, c if M > 1 else (N + 7) // 8 * 8,
                         x if kb > 1 else max(M, 1), y if nb > 1 else kb, be if E > 1 else N * K,
                         ye if E > 1 else 0)
    else:
        (M, K), a = _e4m3("A", A, 2)
        (E, N, K2), b = _e4m3("Bt", Bt, 3)
        if K2 != K:
            raise ValueError(f"shapes do not chain: A{tuple(A.shape)} Bt{tuple(Bt.shape)}")
        dt, ldc = _result_rows("C", C, M, N)
        kb = (K + 127) // 128
        lsb, esb = _block_scales("b_scale", b_scale, (E,), (N + 127) // 128, kb)
        s = _fp8_strides(a[0] if M > 1 else K, b[1] if N > 1 else K, ldc, _row_scales("a_scale", a_scale, M, kb), lsb,
                         b[0] if E > 1 else N * K, esb if E > 1 else 0)
    _vector("offsets", offsets, E + 1, (i32,))
    dev = A.get_device()
    if (stream is not None or dev < 0 or Bt.get_device() != dev or C.get_device() != dev
            or a_scale.get_device() != dev or b_scale.get_device() != dev or offsets.get_device() != dev
            or device() != dev):
        dev = _current_device(("A", "Bt", "C", "a_scale", "b_scale", "offsets"), (A, Bt, C, a_scale, b_scale, offsets))
        raw, _ = _launch_stream(stream, dev)
    else:
        raw = raw_stream(dev)
    st = (_lib or load_library()).tile_gemm_run_fp8_experts(h, A.data_ptr(), Bt.data_ptr(), C.data_ptr(), M, N, K, E,
                                                            offsets.data_ptr(), s, a_scale.data_ptr(),
                                                            b_scale.data_ptr(), dt, raw)
    return _result(st, check) if st else Status.OK


def tile_gemm_run_quantize(h, X, Q, scale, form=Quant.ROWS, gate=None, rows=None, stream=None, check: bool = True):
    """Enqueue bf16 X to E4M3 codes Q (M x K, float8_e4m3fn or uint8) and float32
    scales, as the E4M3 products take them. form=Quant.ROWS: scale (M,
    ceil(K / 128)) with rows next to each other; with `gate`, Q is made of
    act(first half of X's columns) * (second half). form=Quant.BLOCKS: scale
    (ceil(M / 128), ceil(K / 128)). `rows`: M int32 row numbers of X."""
    _, _, _, bf16, _, i32, device, raw_stream = _torch_names or _names()
    (M, K), q = _e4m3("Q", Q, 2)
    blocks = form == 2  # Quant.BLOCKS
    if gate is not None:
        if blocks:
            raise ValueError("gate: not with blocks of 128 x 128")
        form = 1  # Quant.GATED_ROWS
    elif form == 1:
        raise ValueError("form=Quant.GATED_ROWS needs a gate")
    _typed("X", X, bf16)
    x_rows = M
    p_rows = None
    if rows is not None:
        _vector("rows", rows, M, (i32,))
        p_rows = rows.data_ptr()
        if X.dim() == 2:
            x_rows = X.shape[0]
    ldx = _rows_of("X", X, x_rows, K if gate is None else 2 * K)
    kb = (K + 127) // 128
    if blocks:
        lds = _block_scales("scale", scale, (), (M + 127) // 128, kb)[0]
    else:
        lds = _row_scales("scale", scale, M, kb)
    dev = X.get_device()
    if (stream is not None or dev < 0 or Q.get_device() != dev or scale.get_device() != dev
            or (rows is not None and rows.get_device() != dev) or device() != dev):
        dev = _current_device(("X", "Q", "scale", "rows"), (X, Q, scale, rows))
        raw, _ = _launch_stream(stream, dev)
    else:
        raw = raw_stream(dev)
    st = (_lib or load_library()).tile_gemm_run_quantize(h, X.data_ptr(), Q.data_ptr(), scale.data_ptr(), M, K, ldx,
                                                         q[0] if M > 1 else K, lds, form, 0 if gate is None else gate,
                                                         p_rows, x_rows, raw)
    return _result(st, check) if st else Status.OK


def _logits(name, t, T):
    """Experts, type (bfloat16 or not) and row stride of a router's logits of T tokens."""
    names = _torch_names or _names()
    if not isinstance(t, names[0]):
        raise TypeError(f"{name} must be a torch tensor")
    dtype = t.dtype
    bf16 = dtype is names[3]
    if not bf16 and dtype is not names[4]:
        raise TypeError(f"{name} must be float32 or bfloat16, got {dtype}")
    if t.dim() != 2:
        _bad(name, t, f"a row for each of the {T} tokens and a column stride of 1")
    (rows, E), (ld, one) = t.shape, t.stride()
    if rows != T or (one != 1 and E > 1):
        _bad(name, t, f"a row for each of the {T} tokens and a column stride of 1")
    return E, bf16, ld if T > 1 else E


def _per_place(name, t, T, k, dtype):
    """Checks a contiguous (T, k) tensor; its shape."""
    if type(t) is not (_torch_names or _names())[0] or t.dtype is not dtype:
        _typed(name, t, dtype)
    s = t.shape
    if len(s) != 2 or (T is not None and (s[0] != T or s[1] != k)) or not t.is_contiguous():
        _bad(name, t, "contiguous values for each token's experts" if T is None else f"shape ({T}, {k}), contiguous")
    return s


def tile_gemm_run_route(h, logits, ids, weights, score=Score.SOFTMAX, bias=None, groups=1, top_groups=1, group_top=2,
                        renormalize=True, scale=1.0, stream=None, check: bool = True):
    """Enqueue the routing of T tokens: ids (T, k) int32, the k experts of each,
    and weights (T, k) float32, from logits (T, E) float32 or bfloat16. `bias`
    (E float32 values) is added to the scores for the choice only; with groups
    only experts of the top_groups best of `groups` runs of experts are chosen."""
    _, _, _, _, f32, i32, device, raw_stream = _torch_names or _names()
    T, k = _per_place("ids", ids, None, None, i32)
    E, bf16, ld = _logits("logits", logits, T)
    _per_place("weights", weights, T, k, f32)
    p_bias = None
    if bias is not None:
        _vector("bias", bias, E, (f32,))
        p_bias = bias.data_ptr()
    dev = logits.get_device()
    if (stream is not None or dev < 0 or ids.get_device() != dev or weights.get_device() != dev
            or (bias is not None and bias.get_device() != dev) or device() != dev):
        dev = _current_device(("logits", "ids", "weights", "bias"), (logits, ids, weights, bias))
        raw, _ = _launch_stream(stream, dev)
    else:
        raw = raw_stream(dev)
    o = RouteOptions(score, bf16, groups, top_groups, group_top, renormalize, scale)
    st = (_lib or load_library()).tile_gemm_run_route(h, logits.data_ptr(), p_bias, ids.data_ptr(),
                                                      weights.data_ptr(), T, E, k, ld, ctypes.byref(o), raw)
    return _result(st, check) if st else Status.OK


def tile_gemm_run_route_backward(h, logits, ids, dweights, dlogits, score=Score.SOFTMAX, renormalize=True, scale=1.0,
                                 stream=None, check: bool = True):
    """Enqueue the gradient of tile_gemm_run_route's weights: dlogits (T, E, of
    the logits' type) from dweights (T, k) float32 and the ids chosen."""
    _, _, _, _, f32, i32, device, raw_stream = _torch_names or _names()
    T, k = _per_place("ids", ids, None, None, i32)
    E, bf16, ld = _logits("logits", logits, T)
    dE, dbf16, ldd = _logits("dlogits", dlogits, T)
    if dE != E:
        _bad("dlogits", dlogits, f"shape ({T}, {E})")
    if dbf16 != bf16:
        raise TypeError(f"dlogits must be of the logits' type {logits.dtype}, got {dlogits.dtype}")
    _per_place("dweights", dweights, T, k, f32)
    dev = logits.get_device()
    if (stream is not None or dev < 0 or ids.get_device() != dev or dweights.get_device() != dev
            or dlogits.get_device() != dev or device() != dev):
        dev = _current_device(("logits", "ids", "dweights", "dlogits"), (logits, ids, dweights, dlogits))
        raw, _ = _launch_stream(stream, dev)
    else:
        raw = raw_stream(dev)
    o = RouteOptions(score, bf16, 1, 1, 1, renormalize, scale)
    st = (_lib or load_library()).tile_gemm_run_route_backward(h, logits.data_ptr(), ids.data_ptr(),
                                                               dweights.data_ptr(), dlogits.data_ptr(), T, E, k, ld,
                                                               ldd, ctypes.byref(o), raw)
    return _result(st, check) if st else Status.OK


def tile_gemm_place_workspace(T, k, E) -> int:
    """Workspace bytes of tile_gemm_run_place."""
    n = ctypes.c_int64()
    _raise_if(load_library().tile_gemm_place_workspace(T, k, E, ctypes.byref(n)))
    return n.value


def tile_gemm_run_place(h, ids, offsets, rows=None, places=None, first=0, workspace=None, stream=None,
                        check: bool = True):
    """Enqueue the order of the tokens by expert: offsets (E + 1 int32 values,
    E experts from number `first` on), rows (T k) and places (T, k), either of
    which may be left out, from ids (T, k) int32. Without `workspace` one is
    allocated for the call where it needs one."""
    _, _, _, _, _, i32, device, raw_stream = _torch_names or _names()
    T, k = _per_place("ids", ids, None, None, i32)
    _typed("offsets", offsets, i32)
    E = offsets.numel() - 1
    if E < 1 or offsets.dim() != 1 or not offsets.is_contiguous():
        _bad("offsets", offsets, "one dimension of at least 2 contiguous values")
    p_rows = p_places = p_ws = None
    if rows is not None:
        _vector("rows", rows, T * k, (i32,))
        p_rows = rows.data_ptr()
    if places is not None:
        _per_place("places", places, T, k, i32)
        p_places = places.data_ptr()
    dev = ids.get_device()
    if (stream is not None or workspace is not None or dev < 0 or offsets.get_device() != dev
            or (rows is not None and rows.get_device() != dev)
            or (places is not None and places.get_device() != dev) or device() != dev):
        dev = _current_device(("ids", "offsets", "rows", "places", "workspace"),
                              (ids, offsets, rows, places, workspace))
        raw, other = _launch_stream(stream, dev)
    else:
        raw, other = raw_stream(dev), None
    lib = _lib or load_library()
    nbytes = 0
    if workspace is not None:
        nbytes = _workspace_bytes(workspace)
    else:
        n = ctypes.c_int64()
        st = lib.tile_gemm_place_workspace(T, k, E, n)
        if st:
            return _result(st, check)
        nbytes = n.value
        if nbytes:
            workspace = _own_workspace(nbytes, ids, dev, other)
    if workspace is not None:
        p_ws = workspace.data_ptr()
    st = lib.tile_gemm_run_place(h, ids.data_ptr(), T, k, first, E, offsets.data_ptr(), p_rows, p_places, p_ws, nbytes,
                                 raw)
    return _result(st, check) if st else Status.OK


def tile_gemm_run_combine(h, Z, places, weights, Y, stream=None, check: bool = True):
    """Enqueue Y[t] := sum_j weights[t, j] Z[places[t, j]] (Z bf16, Y bf16 or
    float32; places (T, k) int32, those outside Z's rows left out; weights
    (T, k) float32 or None for ones)."""
    tensor, _, _, bf16, f32, i32, device, raw_stream = _torch_names or _names()
    if type(places) is tensor and type(Z) is tensor and type(Y) is tensor and places.dim() == Z.dim() == Y.dim() == 2:
        (T, k), (z_rows, N), (ldz, z1), (ldy, y1), ty = places.shape, Z.shape, Z.stride(), Y.stride(), Y.dtype
        plain = (z1 == y1 == 1 and places.dtype is i32 and places.is_contiguous() and Z.dtype is bf16
                 and (ty is bf16 or ty is f32) and Y.shape == (T, N) and z_rows > 1 and T > 1)
        dt = 1 if ty is bf16 else 0
    else:
        plain = False
    if not plain:
        T, k = _per_place("places", places, None, None, i32)
        z_rows, N = _matrix("Z", Z, None, None)
        ldz = _rows_of("Z", Z, z_rows, N)
        dt, ldy = _result_rows("Y", Y, T, N)
    p_weights = None
    if weights is not None:
        _per_place("weights", weights, T, k, f32)
        p_weights = weights.data_ptr()
    dev = Z.get_device()
    if (stream is not None or dev < 0 or places.get_device() != dev or Y.get_device() != dev
            or (weights is not None and weights.get_device() != dev) or device() != dev):
        dev = _current_device(("Z", "places", "weights", "Y"), (Z, places, weights, Y))
        raw, _ = _launch_stream(stream, dev)
    else:
        raw = raw_stream(dev)
    st = (_lib or load_library()).tile_gemm_run_combine(h, Z.data_ptr(), places.data_ptr(), p_weights, Y.data_ptr(), T,
                                                        N, k, z_rows, ldz, ldy, dt, raw)
    return _result(st, check) if st else Status.OK


def tile_gemm_plan_fp8(M, N, K, experts=0, dtype=Dtype.BF16_TO_BF16, cu_count=256) -> Plan:
    p = Plan()
    _raise_if(load_library().tile_gemm_plan_fp8(int(M), int(N), int(K), int(experts), int(dtype), int(cu_count),
                                                ctypes.byref(p)))
    return p


def tile_gemm_check_mx(A, B, C, M, N, K, strides, a_scale, b_scale, scale_stride, dtype,
                       bias=None, act=Act.NONE, fmt=MX_E4M3) -> Status:
    """Host-only checks of tile_gemm_run_mx's arguments (pointers are integers)."""
    s = strides if isinstance(strides, Strides) else Strides(*strides)
    return Status(load_library().tile_gemm_check_mx(A, B, C, int(M), int(N), int(K), ctypes.byref(s),
                                                    a_scale, b_scale, int(scale_stride), int(fmt),
                                                    int(dtype), bias, int(act)))


def tile_gemm_plan_mx(M, N, K, fmt=0, cu_count=256) -> Plan:
    p = Plan()
    _raise_if(load_library().tile_gemm_plan_mx(int(M), int(N), int(K), int(fmt), int(cu_count),
                                               ctypes.byref(p)))
    return p


def tile_gemm_check_args(A, B, C, M, N, K, strides, dtype) -> Status:
    """Host-only argument checks (pointers are plain integers here)."""
    s = strides if isinstance(strides, Strides) else Strides(*strides)
    return Status(load_library().tile_gemm_check_args(A, B, C, int(M), int(N), int(K),
                                                      ctypes.byref(s), int(dtype)))


def tile_gemm_check_epilogue(C, M, N, strides, dtype, bias, act) -> Status:
    """Host-only checks of the fused epilogue's arguments."""
    s = strides if isinstance(strides, Strides) else Strides(*strides)
    return Status(load_library().tile_gemm_check_epilogue(C, int(M), int(N), ctypes.byref(s),
                                                          int(dtype), bias, int(act)))


def tile_gemm_plan(M, N, K, b_col_major=False, cu_count=256) -> Plan:
    p = Plan()
    _raise_if(load_library().tile_gemm_plan(int(M), int(N), int(K), int(bool(b_col_major)),
                                            int(cu_count), ctypes.byref(p)))
    return p


def tile_gemm_tile_of(plan: Plan, M, N, wg):
    vals = [ctypes.c_int64() for _ in range(4)]
    _raise_if(load_library().tile_gemm_tile_of(ctypes.byref(plan), int(M), int(N), int(wg),
                                               *[ctypes.byref(v) for v in vals]))
    return tuple(v.value for v in vals)


class TileGemm:
    """Owns one handle; ``g(A, B, C)`` enqueues C := A.B on the current stream."""

    def __init__(self, device: int = 0):
        self.handle = tile_gemm_create(device)

    def __call__(self, A, B, C, stream=None, bias=None, act=None):
        if bias is None and act is None:
            return tile_gemm_run(self.handle, A, B, C, stream=stream)
        return tile_gemm_run_epilogue(self.handle, A, B, C, bias=bias,
                                      act=Act.NONE if act is None else act, stream=stream)

    def run_debug(self, A, B, C, counts=None, flags=0, stream=None, bias=None, act=None):
        return tile_gemm_run_debug(self.handle, A, B, C, counts=counts, flags=flags,
                                   stream=stream, bias=bias,
                                   act=Act.NONE if act is None else act)

    def mx(self, A, Bt, C, a_scale, b_scale, bias=None, act=None, stream=None, counts=None,
           flags=0, fmt=MX_E4M3):
        """MX product (tile_gemm_run_mx) into C."""
        return tile_gemm_run_mx(self.handle, A, Bt, C, a_scale, b_scale, bias=bias,
                                act=Act.NONE if act is None else act, stream=stream,
                                counts=counts, flags=flags, fmt=fmt)

    def glu(self, A, B, C, gate=Gate.SILU, bias=None, stream=None):
        """Gated block (tile_gemm_run_glu) into C."""
        return tile_gemm_run_glu(self.handle, A, B, C, gate=gate, bias=bias, stream=stream)

    def glu_backward(self, A, B, dC, dA=None, dB=None, gate=Gate.SILU, bias=None, dbias=None,
                     workspace=None, stream=None):
        """Backward pass of the gated block (tile_gemm_run_glu_backward)."""
        return tile_gemm_run_glu_backward(self.handle, A, B, dC, dA=dA, dB=dB, gate=gate, bias=bias,
                                          dbias=dbias, workspace=workspace, stream=stream)

    def xent(self, A, B, target, loss=None, lse=None, ignore_index=-100, label_smoothing=0.0,
             z_loss=0.0, workspace=None, stream=None):
        """Cross entropy of the projection A.B (tile_gemm_run_xent)."""
        return tile_gemm_run_xent(self.handle, A, B, target, loss=loss, lse=lse,
                                  ignore_index=ignore_index, label_smoothing=label_smoothing,
                                  z_loss=z_loss, workspace=workspace, stream=stream)

    def xent_backward(self, A, B, target, lse, dloss, dA=None, dB=None, ignore_index=-100,
                      label_smoothing=0.0, z_loss=0.0, piece=0, workspace=None, stream=None):
        """Gradients of the cross entropy (tile_gemm_run_xent_backward)."""
        return tile_gemm_run_xent_backward(self.handle, A, B, target, lse, dloss, dA=dA, dB=dB,
                                           ignore_index=ignore_index, label_smoothing=label_smoothing,
                                           z_loss=z_loss, piece=piece, workspace=workspace, stream=stream)

    def fp8(self, A, Bt, C, a_scale, b_scale, bias=None, act=None, stream=None):
        """E4M3 product with block scales (tile_gemm_run_fp8) into C."""
        return tile_gemm_run_fp8(self.handle, A, Bt, C, a_scale, b_scale, bias=bias,
                                 act=Act.NONE if act is None else act, stream=stream)

    def fp8_experts(self, A, Bt, C, a_scale, b_scale, offsets, stream=None):
        """The same over rows sorted by expert (tile_gemm_run_fp8_experts)."""
        return tile_gemm_run_fp8_experts(self.handle, A, Bt, C, a_scale, b_scale, offsets, stream=stream)

    def quantize(self, X, Q, scale, form=Quant.ROWS, gate=None, rows=None, stream=None):
        """bf16 to E4M3 and scales (tile_gemm_run_quantize)."""
        return tile_gemm_run_quantize(self.handle, X, Q, scale, form=form, gate=gate, rows=rows, stream=stream)

    def route(self, logits, ids, weights, score=Score.SOFTMAX, bias=None, groups=1, top_groups=1, group_top=2,
              renormalize=True, scale=1.0, stream=None):
        """Experts of each token and their weights (tile_gemm_run_route)."""
        return tile_gemm_run_route(self.handle, logits, ids, weights, score=score, bias=bias, groups=groups,
                                   top_groups=top_groups, group_top=group_top, renormalize=renormalize,
                                   scale=scale, stream=stream)

    def route_backward(self, logits, ids, dweights, dlogits, score=Score.SOFTMAX, renormalize=True, scale=1.0,
                       stream=None):
        """Gradient of the routing weights (tile_gemm_run_route_backward)."""
        return tile_gemm_run_route_backward(self.handle, logits, ids, dweights, dlogits, score=score,
                                            renormalize=renormalize, scale=scale, stream=stream)

    def place(self, ids, offsets, rows=None, places=None, first=0, workspace=None, stream=None):
        """The tokens' order by expert (tile_gemm_run_place)."""
        return tile_gemm_run_place(self.handle, ids, offsets, rows=rows, places=places, first=first,
                                   workspace=workspace, stream=stream)

    def combine(self, Z, places, weights, Y, stream=None):
        """Weighted sums of the experts' rows (tile_gemm_run_combine)."""
        return tile_gemm_run_combine(self.handle, Z, places, weights, Y, stream=stream)

    def close(self):
        if self.handle is not None:
            tile_gemm_destroy(self.handle)
            self.handle = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):  # pragma: no cover - best effort
        try:
            self.close()
        except Exception:
            pass
