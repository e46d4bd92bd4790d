"""Python binding of libfusedmx.so (argument marshalling only).

The operators that consume MXFP4 rows (include/fusedmx.h): `gemm`,
`grouped_gemm`, `silu_mul_quant` and `combine` take torch CUDA tensors as
mxfp4_quantization_b200.fusednorm returns them, allocate the outputs with torch,
call the C ABI on the current stream of the tensors' device, and raise
`FusedMXError` on a non-zero status.  `mx_gemm`, `mx_grouped_gemm`,
`mx_silu_mul_quant` and `mx_combine` are the C ABI one to one.

Scales are told apart by their shape, as fusednorm.alloc_outputs makes them:
[rows, K/32] is row-major, a flat buffer is the 32x4x4 tiling
(FN_SCALE_SWIZZLE_32_4_4).

The operators are for inference: outputs carry no gradient, whatever the inputs
require.

There is no fallback: if the library is missing, importing this module fails.
"""
import ctypes
import math
import os
from collections import namedtuple
from functools import lru_cache
from typing import Optional, Union

import torch

from .fusednorm import (FN_FP8_PER_GROUP128, FN_FP8_PER_TOKEN, FN_IO_FP16, FN_MODE_MASK, FN_MXFP4, FN_OK,
                        FN_SCALE_MN_MAJOR, FN_SCALE_SWIZZLE_32_4_4, MODES, alloc_outputs)

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfusedmx.so")

MX_OUT_BF16 = 0x0
MX_OUT_FP16 = 0x1
MX_OUT_FP32 = 0x2
MX_A_SCALE_SWIZZLE = 0x10
MX_B_SCALE_SWIZZLE = 0x20
MX_MAX_EXPERTS = 1024
MX_MAX_TOP = 32
MX_SMALL_ROWS = 64
MX_SMALL_EXPERT_ROWS = 16

MX_VARIANT_NONE = 0
MX_VARIANT_GEMM = 1
MX_VARIANT_SILU_GROUPS = 2
MX_VARIANT_SILU_ROW = 3
MX_VARIANT_COMBINE = 4
MX_VARIANT_COMBINE_NARROW = 5
MX_VARIANT_GEMM_PAIR = 6

OUT_FLAGS = {torch.bfloat16: MX_OUT_BF16, torch.float16: MX_OUT_FP16, torch.float32: MX_OUT_FP32}

# The exported symbols of include/fusedmx.h.
ABI_SYMBOLS = ("mx_gemm", "mx_gemm_workspace_bytes", "mx_grouped_gemm",
               "mx_grouped_gemm_workspace_bytes", "mx_silu_mul_quant", "mx_combine",
               "mx_last_variant", "mx_last_launch", "mx_programmatic_launch",
               "mx_status_string", "mx_version")


class FusedMXError(RuntimeError):
    def __init__(self, func: str, status: int):
        super().__init__(f"{func}: {mx_status_string(status)} (status {status})")
        self.status = status


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is not built; run `python -m mxfp4_quantization_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.mx_gemm.argtypes = [vp, vp, vp, vp, i64, i64, i64, i32, vp, i64, vp, vp]
    lib.mx_gemm.restype = i32
    lib.mx_gemm_workspace_bytes.argtypes = [i64, i64, i64, i32]
    lib.mx_gemm_workspace_bytes.restype = i64
    lib.mx_grouped_gemm.argtypes = [vp, vp, i64, vp, vp, i64, vp, vp, i64, i64, i64, i32, vp, i64,
                                    vp, vp]
    lib.mx_grouped_gemm.restype = i32
    lib.mx_grouped_gemm_workspace_bytes.argtypes = [i64, i64, i64, i64, i32, i32]
    lib.mx_grouped_gemm_workspace_bytes.restype = i64
    lib.mx_silu_mul_quant.argtypes = [vp, i64, i32, i64, i64, vp, vp, vp, vp, vp]
    lib.mx_silu_mul_quant.restype = i32
    lib.mx_combine.argtypes = [vp, i64, vp, vp, vp, i64, i32, i64, i32, vp, vp]
    lib.mx_combine.restype = i32
    lib.mx_last_variant.argtypes = []
    lib.mx_last_variant.restype = i32
    lib.mx_last_launch.argtypes = [ctypes.POINTER(ctypes.c_int32)]
    lib.mx_last_launch.restype = None
    lib.mx_programmatic_launch.argtypes = [i32]
    lib.mx_programmatic_launch.restype = i32
    lib.mx_status_string.argtypes = [i32]
    lib.mx_status_string.restype = ctypes.c_char_p
    lib.mx_version.argtypes = []
    lib.mx_version.restype = i32
    return lib


_lib = _load()


# ---- the C ABI, one to one --------------------------------------------------------


def mx_gemm(a_q, a_scale, b_q, b_scale, M: int, N: int, K: int, flags: int, out, ldo: int,
            workspace, stream: Optional[int]) -> int:
    return _lib.mx_gemm(a_q, a_scale, b_q, b_scale, M, N, K, flags, out, ldo, workspace, stream)


def mx_gemm_workspace_bytes(M: int, N: int, K: int, flags: int) -> int:
    return _lib.mx_gemm_workspace_bytes(M, N, K, flags)


def mx_grouped_gemm(a_q, a_scale, a_rows: int, rows, offsets, E: int, b_q, b_scale, R: int, N: int,
                    K: int, flags: int, out, ldo: int, workspace,
                    stream: Optional[int]) -> int:
    return _lib.mx_grouped_gemm(a_q, a_scale, a_rows, rows, offsets, E, b_q, b_scale, R, N, K,
                                flags, out, ldo, workspace, stream)


def mx_grouped_gemm_workspace_bytes(R: int, E: int, N: int, K: int, flags: int,
                                    gather: int) -> int:
    return _lib.mx_grouped_gemm_workspace_bytes(R, E, N, K, flags, gather)


def mx_silu_mul_quant(x, ldx: int, mode: int, M: int, H: int, num_rows, out_q, out_scale, out_y,
                      stream: Optional[int]) -> int:
    return _lib.mx_silu_mul_quant(x, ldx, mode, M, H, num_rows, out_q, out_scale, out_y, stream)


def mx_combine(y, R: int, pos, weight, base, T: int, k: int, N: int, flags: int, out,
               stream: Optional[int]) -> int:
    return _lib.mx_combine(y, R, pos, weight, base, T, k, N, flags, out, stream)


def mx_last_variant() -> int:
    return _lib.mx_last_variant()


def mx_last_launch():
    out = (ctypes.c_int32 * 4)()
    _lib.mx_last_launch(out)
    return tuple(out)


def mx_programmatic_launch(on: int) -> int:
    return _lib.mx_programmatic_launch(on)


def mx_status_string(status: int) -> str:
    return _lib.mx_status_string(status).decode()


def mx_version() -> int:
    return _lib.mx_version()


class programmatic_launch:
    """Context manager: this thread's calls launch their kernels as
    programmatic dependents of the stream's previous work (see
    fn_programmatic_launch)."""

    def __init__(self, on: bool = True):
        self.on = on

    def __enter__(self):
        self.old = mx_programmatic_launch(1 if self.on else 0)
        return self

    def __exit__(self, *exc):
        mx_programmatic_launch(self.old)
        return False


# ---- tensor API ----------------------------------------------------------------------

SiluMulQuantOutput = namedtuple("SiluMulQuantOutput", "q scale y")


# A decode step makes these calls every few microseconds.  Each first tests what
# every good call has in one expression (dtype, device number, contiguity: what is
# cheapest to read); only where that fails the checks that name the fault run.

_U8, _I32, _F32 = torch.uint8, torch.int32, torch.float32
_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def _call(func, i: int, *args) -> int:
    """func(*args, stream) on the current stream of device number i, with that
    device current."""
    if i == _current_device():
        return func(*args, _raw_stream(i))
    with torch.cuda.device(i):
        return func(*args, _raw_stream(i))


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _round_up(x: int, m: int) -> int:
    return (x + m - 1) // m * m


def _tensor(t: torch.Tensor, name: str, dtype, dim=None, device=None) -> torch.Tensor:
    """A contiguous CUDA tensor of `dtype` on the call's device."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if dim is not None and t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions, got {t.dim()}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call on {device}")
    return t


def _scale_fault(t: torch.Tensor, name: str, lead: int, rows: int, G: int, device):
    """Raises for scales that are neither [rows, G] nor the 32x4x4 tiling (per
    expert, if lead is the number of experts and not 0)."""
    if t.dtype is not _U8 and t.dtype is not torch.float8_e8m0fnu:
        raise TypeError(f"{name} must be uint8 (E8M0 bytes), got {t.dtype}")
    if not t.is_cuda or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous tensor on {device}")
    first = f"{lead}, " if lead else ""
    raise ValueError(f"{name} has shape {tuple(t.shape)}: expected ({first}{rows}, {G}), or "
                     f"({first}{_round_up(rows, 128) * _round_up(G, 4)}) in the 32x4x4 tiling")


def _tiled(t: torch.Tensor, name: str, lead: int, rows: int, G: int, i: int, device) -> bool:
    """Whether E8M0 scales of `rows` rows of G groups are in the 32x4x4 tiling (flat
    per expert) or row-major; raises where they are neither."""
    if (t.dtype is _U8 or t.dtype is torch.float8_e8m0fnu) and t.get_device() == i and \
            t.is_contiguous():
        shape = t.shape
        n = len(shape) - (1 if lead else 0)
        if n == 2:
            if shape[-1] == G and shape[-2] == rows and (not lead or shape[0] == lead):
                return False
        elif n == 1:
            if shape[-1] == _round_up(rows, 128) * _round_up(G, 4) and \
                    (not lead or shape[0] == lead):
                return True
    _scale_fault(t, name, lead, rows, G, device)


def _product_out(out, out_dtype, M: int, N: int, device):
    """The output tensor, its flag and its row stride."""
    if out is None:
        flag = OUT_FLAGS.get(out_dtype)
        if flag is None:
            raise TypeError(f"out_dtype must be bfloat16, float16 or float32, got {out_dtype}")
        # (the quickest of torch's allocating calls)
        return torch.empty_strided((M, N), (N, 1), dtype=out_dtype, device=device), flag, N
    if out.device != device:
        raise ValueError(f"out must be on {device}")
    flag = OUT_FLAGS.get(out.dtype)
    if flag is None:
        raise TypeError(f"out must be bfloat16, float16 or float32, got {out.dtype}")
    if out.shape != (M, N):
        raise ValueError(f"out has shape {tuple(out.shape)}, expected {(M, N)}")
    ldo, step = out.stride()
    if M <= 1:
        ldo = max(N, ldo)
    if (N > 1 and step != 1) or ldo < N:
        raise ValueError("out needs a contiguous last dim and rows that do not overlap")
    return out, flag, ldo


# (sizes and flags only; a few hundred different ones in a program)
_gemm_bytes = lru_cache(maxsize=1024)(lambda *a: _lib.mx_gemm_workspace_bytes(*a))
_grouped_bytes = lru_cache(maxsize=1024)(lambda *a: _lib.mx_grouped_gemm_workspace_bytes(*a))


def _workspace(need: int, given: Optional[torch.Tensor], device):
    """The call's workspace: `given`, or one from torch's allocator."""
    if need <= 0:
        return None
    if given is None:
        return torch.empty_strided((need,), (1,), dtype=_U8, device=device)
    if given.device != device or not given.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    if given.numel() * given.element_size() < need:
        raise ValueError(f"workspace holds fewer than the {need} bytes the call needs")
    return given


def gemm(a_q: torch.Tensor, a_scale: torch.Tensor, b_q: torch.Tensor, b_scale: torch.Tensor, *,
         out: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
         workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out[m, n] = sum_k a[m, k] b[n, k] of two MXFP4 operands: codes uint8
    [M, K/2] and [N, K/2], scales as quant and rmsnorm_quant return them
    (row-major or in the 32x4x4 tiling).  `out` may have any row stride; its
    type, else `out_dtype`, is the output type (bfloat16, float16, float32).  The
    workspace (mx_gemm_workspace_bytes) is allocated with torch unless given."""
    i = a_q.get_device()
    if i < 0 or a_q.dtype is not _U8 or b_q.dtype is not _U8 or b_q.get_device() != i or \
            a_q.dim() != 2 or b_q.dim() != 2 or not a_q.is_contiguous() or \
            not b_q.is_contiguous():
        _tensor(a_q, "a_q", _U8, 2)
        _tensor(b_q, "b_q", _U8, 2, a_q.device)
    M, half = a_q.shape
    N, other = b_q.shape
    if half != other:
        raise ValueError(f"a_q rows have {2 * half} codes, b_q rows {2 * other}")
    dev = a_q.device
    flags = MX_A_SCALE_SWIZZLE if _tiled(a_scale, "a_scale", 0, M, half // 16, i, dev) else 0
    if _tiled(b_scale, "b_scale", 0, N, half // 16, i, dev):
        flags |= MX_B_SCALE_SWIZZLE
    out, f, ldo = _product_out(out, out_dtype, M, N, dev)
    flags |= f
    ws = None
    if M > MX_SMALL_ROWS:
        ws = _workspace(_gemm_bytes(M, N, 2 * half, flags), workspace, dev)
    st = _call(_lib.mx_gemm, i, a_q.data_ptr(), a_scale.data_ptr(), b_q.data_ptr(),
               b_scale.data_ptr(), M, N, 2 * half, flags, out.data_ptr(), ldo, _ptr(ws))
    if st != FN_OK:
        raise FusedMXError("mx_gemm", st)
    return out


def grouped_gemm(a_q: torch.Tensor, a_scale: torch.Tensor, b_q: torch.Tensor,
                 b_scale: torch.Tensor, offsets: torch.Tensor, *,
                 rows: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                 out_dtype: torch.dtype = torch.bfloat16,
                 workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """gemm with one weight per expert: b_q uint8 [E, N, K/2], b_scale
    [E, N, K/32] or [E, bytes of one 32x4x4 tiling]; expert e computes the
    rows offsets[e] <= r < offsets[e+1] (int32 [E+1] on the device) of out
    from the rows `rows[r]` (int32 [R]) of a, or from row r itself.  out has
    as many rows as `rows`, else as a_q (an out that is given may have fewer:
    the ranges end there); rows that no expert owns keep what they held (a new
    out is not filled)."""
    i = a_q.get_device()
    if i < 0 or a_q.dtype is not _U8 or b_q.dtype is not _U8 or offsets.dtype is not _I32 or \
            b_q.get_device() != i or offsets.get_device() != i or a_q.dim() != 2 or \
            b_q.dim() != 3 or offsets.dim() != 1 or not a_q.is_contiguous() or \
            not b_q.is_contiguous() or not offsets.is_contiguous():
        _tensor(a_q, "a_q", _U8, 2)
        _tensor(b_q, "b_q", _U8, 3, a_q.device)
        _tensor(offsets, "offsets", _I32, 1, a_q.device)
    a_rows, half = a_q.shape
    E, N, other = b_q.shape
    if half != other:
        raise ValueError(f"a_q rows have {2 * half} codes, b_q rows {2 * other}")
    if offsets.shape[0] != E + 1:
        raise ValueError(f"offsets has {offsets.shape[0]} entries, expected {E + 1}")
    dev = a_q.device
    if _tiled(a_scale, "a_scale", 0, a_rows, half // 16, i, dev):
        raise ValueError("a_scale must be row-major [rows, K/32] for ragged row ranges")
    flags = MX_B_SCALE_SWIZZLE if _tiled(b_scale, "b_scale", E, N, half // 16, i, dev) else 0
    if rows is not None:
        R = _tensor(rows, "rows", _I32, 1, dev).shape[0]
    else:
        R = a_rows if out is None else min(a_rows, out.shape[0])
    out, f, ldo = _product_out(out, out_dtype, R, N, dev)
    flags |= f
    ws = None
    if R > MX_SMALL_EXPERT_ROWS * E:
        ws = _workspace(_grouped_bytes(R, E, N, 2 * half, flags, 0 if rows is None else 1),
                        workspace, dev)
    st = _call(_lib.mx_grouped_gemm, i, a_q.data_ptr(), a_scale.data_ptr(), a_rows, _ptr(rows),
               offsets.data_ptr(), E, b_q.data_ptr(), b_scale.data_ptr(), R, N, 2 * half, flags,
               out.data_ptr(), ldo, _ptr(ws))
    if st != FN_OK:
        raise FusedMXError("mx_grouped_gemm", st)
    return out


def silu_mul_quant(x: torch.Tensor, mode: Union[int, str], *,
                   num_rows: Optional[torch.Tensor] = None, emit_y: bool = False,
                   out_q: Optional[torch.Tensor] = None,
                   out_scale: Optional[torch.Tensor] = None,
                   out_y: Optional[torch.Tensor] = None) -> SiluMulQuantOutput:
    """y = silu(gate) * up of bf16 (or float16) rows [..., 2H] = [gate | up],
    rounded once to 16 bits, and its quantization (mode as fusednorm.quant's);
    returns (q, scale, y), y None unless `emit_y` (or `out_y`) asks for it.  A
    2-D x may have any row stride that is a multiple of 8 elements.  `num_rows`
    (int32 [1] on the device): only the first *num_rows rows are computed."""
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    dt = x.dtype
    m = MODES[mode] if isinstance(mode, str) else int(mode)
    if dt is torch.float16:
        m |= FN_IO_FP16
    elif dt is not torch.bfloat16:
        raise TypeError(f"x must be bfloat16 or float16, got {dt}")
    elif m & FN_IO_FP16:
        raise TypeError("FN_IO_FP16 was asked for but the rows are bfloat16")
    if x.dim() != 2:
        if not x.is_contiguous() or x.dim() == 0:
            raise ValueError("x must be contiguous, or 2-D with a contiguous last dim")
        x = x.reshape(math.prod(x.shape[:-1]), x.shape[-1])
    M, H = x.shape
    if H % 2:
        raise ValueError("x rows hold a gate half and an up half: an even last dim")
    ldx, step = x.stride()
    if step != 1 and H > 1:
        raise ValueError("x needs a contiguous last dim")
    if M <= 1:
        ldx = H
    H //= 2
    dev = x.device
    if num_rows is not None and _tensor(num_rows, "num_rows", torch.int32, None, dev).numel() != 1:
        raise ValueError("num_rows must hold one value")
    if out_q is None and out_scale is None:
        out_q, out_scale = _alloc_quant(m, M, H, dev)
    else:
        if out_q is None or out_scale is None:
            q, s = alloc_outputs(m, M, H, dev)
            out_q = q if out_q is None else out_q
            out_scale = s if out_scale is None else out_scale
        _check_quant(out_q, out_scale, m, M, H, dev)
    if out_y is None and emit_y:
        out_y = torch.empty_strided((M, H), (H, 1), dtype=dt, device=dev)
    elif out_y is not None:
        if _tensor(out_y, "out_y", dt, None, dev).numel() != M * H:
            raise ValueError(f"out_y must hold {M} x {H} values")
    st = _call(_lib.mx_silu_mul_quant, dev.index, x.data_ptr(), ldx, m, M, H, _ptr(num_rows),
               out_q.data_ptr(), out_scale.data_ptr(), _ptr(out_y))
    if st != FN_OK:
        raise FusedMXError("mx_silu_mul_quant", st)
    return SiluMulQuantOutput(out_q, out_scale, out_y)


def _alloc_quant(mode: int, M: int, H: int, device):
    """fusednorm.alloc_outputs, for row-major scales by torch's quickest call."""
    kind = mode & ~FN_IO_FP16
    if kind == FN_MXFP4:
        dt, w, sdt, g = _U8, H // 2, _U8, H // 32
    elif kind == FN_FP8_PER_TOKEN:
        dt, w, sdt, g = torch.float8_e4m3fn, H, _F32, 1
    elif kind == FN_FP8_PER_GROUP128:
        dt, w, sdt, g = torch.float8_e4m3fn, H, _F32, H // 128
    else:
        return alloc_outputs(mode, M, H, device)
    return (torch.empty_strided((M, w), (w, 1), dtype=dt, device=device),
            torch.empty_strided((M, g), (g, 1), dtype=sdt, device=device))


def _check_quant(q, scale, mode: int, M: int, H: int, device):
    """Outputs that the caller brought are large enough."""
    kind = mode & FN_MODE_MASK
    if kind == FN_MXFP4:
        codes = M * H // 2
        scales = _round_up(M, 128) * _round_up(H // 32, 4) if mode & FN_SCALE_SWIZZLE_32_4_4 \
            else M * (H // 32)
    else:
        codes = M * H
        scales = 4 * (M if kind == FN_FP8_PER_TOKEN else
                      (_round_up(M, 4) if mode & FN_SCALE_MN_MAJOR else M) * (H // 128))
    for t, n, name in ((q, codes, "out_q"), (scale, scales, "out_scale")):
        if not t.is_cuda or t.device != device or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous tensor on {device}")
        if t.numel() * t.element_size() < n:
            raise ValueError(f"{name} holds fewer than {n} bytes")


def combine(y: torch.Tensor, pos: torch.Tensor, weight: torch.Tensor, *,
            base: Optional[torch.Tensor] = None,
            out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out[t] = base[t] + sum_j weight[t, j] y[pos[t, j]]: y bf16 (or float16)
    [R, N], pos int32 [T, k] (positions outside [0, R) are skipped), weight
    fp32 [T, k], base and out of y's type [T, N] (out may be base)."""
    dt, i = y.dtype, y.get_device()
    if dt is not torch.bfloat16 and dt is not torch.float16:
        raise TypeError(f"y must be bfloat16 or float16, got {dt}")
    if i < 0 or pos.dtype is not _I32 or weight.dtype is not _F32 or pos.get_device() != i or \
            weight.get_device() != i or y.dim() != 2 or pos.dim() != 2 or \
            not y.is_contiguous() or not pos.is_contiguous() or not weight.is_contiguous():
        _tensor(y, "y", dt, 2)
        _tensor(pos, "pos", _I32, 2, y.device)
        _tensor(weight, "weight", _F32, 2, y.device)
    R, N = y.shape
    T, k = pos.shape
    if weight.shape != pos.shape:
        raise ValueError(f"weight has shape {tuple(weight.shape)}, pos {tuple(pos.shape)}")
    if base is not None and _tensor(base, "base", dt, 2, y.device).shape != (T, N):
        raise ValueError(f"base has shape {tuple(base.shape)}, expected {(T, N)}")
    if out is None:
        out = torch.empty_strided((T, N), (N, 1), dtype=dt, device=y.device)
    elif _tensor(out, "out", dt, 2, y.device).shape != (T, N):
        raise ValueError(f"out has shape {tuple(out.shape)}, expected {(T, N)}")
    st = _call(_lib.mx_combine, i, y.data_ptr(), R, pos.data_ptr(), weight.data_ptr(),
               _ptr(base), T, k, N, FN_IO_FP16 if dt is torch.float16 else 0, out.data_ptr())
    if st != FN_OK:
        raise FusedMXError("mx_combine", st)
    return out
