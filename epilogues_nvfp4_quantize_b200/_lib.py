"""ctypes binding of libnvfp4epi.so: argument marshalling only.

Every computation runs in the library's CUDA kernels; this module turns torch tensors
into device pointers, sizes and the current stream, and raises RuntimeError on a
non-OK status. There is no CPU fallback: if the shared library is missing or cannot
be loaded, every call fails loudly.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libnvfp4epi.so")

SWIGLU_INTERLEAVE = 1

# Entry points declared in include/nvfp4epi.h (kept in sync by tests/test_abi.py).
EXPORTS = (
    "nvfp4_sf_bytes", "nvfp4_quantize_workspace_bytes", "nvfp4_quantize",
    "gemm_nvfp4_plain", "gemm_nvfp4_rmsnorm", "gemm_nvfp4_swiglu",
    "rmsnorm_heads_bf16", "swiglu_bf16", "nvfp4_status_string",
    "nvfp4_read_device_status", "nvfp4_selftest_bounded_wait", "nvfp4_launch_count",
    "nvfp4_quantize_noalloc", "nvfp4_fake_quantize", "gemm_nvfp4_pointwise",
    "mxfp4_sf_bytes", "mxfp4_quantize", "gemm_mxfp4_pointwise", "gemm_mxfp4_plain",
    "gemm_mxfp4_rmsnorm", "gemm_mxfp4_swiglu", "gemm_nvfp4_reduce_rows_f32", "nvfp4_signal_barrier",
    "gemv_nvfp4", "residual_norm", "residual_norm_backward", "residual_norm_workspace_bytes", "rope_axes",
)


class _Tensor(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("sf", ctypes.c_void_p), ("gscale", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64)]


_lib = None


def load() -> ctypes.CDLL:
    """Load the shared library (once). Raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libnvfp4epi.so not built at {LIB_PATH}; run __graft_entry__.build()")
    lib = ctypes.CDLL(LIB_PATH)
    i64, vp, i32, f32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    sig = {
        "nvfp4_sf_bytes": (i64, [i64, i64]),
        "nvfp4_quantize_workspace_bytes": (i64, []),
        "nvfp4_quantize": (i32, [vp, i64, i64, i64, i32, i32, _Tensor, vp, vp]),
        "gemm_nvfp4_plain": (i32, [_Tensor, _Tensor, vp, i64, vp]),
        "gemm_nvfp4_rmsnorm": (i32, [_Tensor, _Tensor, vp, i32, i64, f32, vp, i64, vp]),
        "gemm_nvfp4_swiglu": (i32, [_Tensor, _Tensor, vp, i64, ctypes.POINTER(_Tensor), vp]),
        "rmsnorm_heads_bf16": (i32, [vp, i64, i64, vp, i32, i64, f32, vp, i64, vp]),
        "swiglu_bf16": (i32, [vp, i64, i64, i64, vp, i64, vp]),
        "nvfp4_status_string": (ctypes.c_char_p, [i32]),
        "nvfp4_read_device_status": (i32, [vp]),
        "nvfp4_selftest_bounded_wait": (i32, [i64, vp]),
        "nvfp4_launch_count": (i64, []),
        "nvfp4_quantize_noalloc": (i32, [vp, i64, i64, i64, i32, _Tensor, vp]),
        "nvfp4_fake_quantize": (i32, [vp, i64, i64, i64, i32, vp, vp, i64, vp, vp]),
        "gemm_nvfp4_pointwise": (i32, [_Tensor, _Tensor, vp, i32, i32, vp, i64, ctypes.POINTER(_Tensor), vp]),
        "gemm_nvfp4_reduce_rows_f32": (i32, [_Tensor, _Tensor, vp, i32, i64, i64, vp]),
        "mxfp4_sf_bytes": (i64, [i64, i64]),
        "mxfp4_quantize": (i32, [vp, i64, i64, i64, i32, _Tensor, vp]),
        "gemm_mxfp4_pointwise": (i32, [_Tensor, _Tensor, vp, i32, i32, vp, i64, vp]),
        "gemm_mxfp4_plain": (i32, [_Tensor, _Tensor, vp, i64, vp]),
        "gemm_mxfp4_rmsnorm": (i32, [_Tensor, _Tensor, vp, i32, i64, f32, vp, i64, vp]),
        "gemm_mxfp4_swiglu": (i32, [_Tensor, _Tensor, vp, i64, ctypes.POINTER(_Tensor), vp]),
        "nvfp4_signal_barrier": (i32, [vp, i32, i32, ctypes.c_uint32, i64, vp]),
        "gemv_nvfp4": (i32, [vp, i32, i64, i64, i32, _Tensor, vp, i32, vp, i64, vp]),
        "residual_norm": (i32, [ctypes.c_char_p, vp, i64, vp, i64, ctypes.POINTER(_Tensor), vp, vp]),
        "residual_norm_workspace_bytes": (i64, [i64, i64, i64]),
        "residual_norm_backward": (i32, [ctypes.c_char_p, vp, ctypes.c_char_p, vp, vp]),
        "rope_axes": (i32, [vp, i32, i64, i64, i64, i64, i64, vp, i32, i64, i32, ctypes.POINTER(ctypes.c_int32), vp,
                            i32, i32, vp, i64, i64, vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(status: int, what: str) -> None:
    if status != 0:
        msg = load().nvfp4_status_string(status).decode()
        raise RuntimeError(f"{what}: {msg} (status {status})")


def _stream(stream) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


class NVFP4Tensor:
    """Device buffers of an NVFP4 tensor (see nvfp4_tensor in include/nvfp4epi.h)."""

    def __init__(self, codes: torch.Tensor, sf: torch.Tensor, gscale: torch.Tensor, rows: int, cols: int):
        self.codes, self.sf, self.gscale, self.rows, self.cols = codes, sf, gscale, rows, cols

    @classmethod
    def empty(cls, rows: int, cols: int, device="cuda") -> "NVFP4Tensor":
        return cls(torch.empty((rows, cols // 2), dtype=torch.uint8, device=device),
                   torch.empty((sf_bytes(rows, cols),), dtype=torch.uint8, device=device),
                   torch.empty((1,), dtype=torch.float32, device=device), rows, cols)

    @classmethod
    def empty_mx(cls, rows: int, cols: int, device="cuda") -> "NVFP4Tensor":
        """Buffers of an MXFP4 tensor (E8M0 scales per 32 values; see mxfp4_quantize)."""
        return cls(torch.empty((rows, cols // 2), dtype=torch.uint8, device=device),
                   torch.empty((int(load().mxfp4_sf_bytes(rows, cols)),), dtype=torch.uint8, device=device),
                   torch.empty((1,), dtype=torch.float32, device=device), rows, cols)

    def c(self) -> _Tensor:
        return _Tensor(self.codes.data_ptr(), self.sf.data_ptr(), self.gscale.data_ptr(), self.rows, self.cols)

    def nbytes(self) -> int:
        return self.codes.numel() + self.sf.numel() + 4


def sf_bytes(rows: int, cols: int) -> int:
    return int(load().nvfp4_sf_bytes(rows, cols))


def quantize_workspace_bytes() -> int:
    return int(load().nvfp4_quantize_workspace_bytes())


def _check_workspace(workspace: torch.Tensor, need: int) -> None:
    """A workspace has to own the bytes that its size says (an expanded tensor does not)."""
    if not workspace.is_contiguous() or workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace holds {workspace.numel() * workspace.element_size()} bytes, needs {need} contiguous ones")


def _workspace(workspace: Optional[torch.Tensor], compute_amax: bool, device) -> Optional[torch.Tensor]:
    """The caller's workspace (checked for size), or a new one when none is given."""
    if not compute_amax:
        return workspace
    need = quantize_workspace_bytes()
    if workspace is None:
        return torch.empty((need,), dtype=torch.uint8, device=device)
    _check_workspace(workspace, need)
    return workspace


def nvfp4_quantize(x: torch.Tensor, out: NVFP4Tensor, compute_amax: bool = True, interleave: bool = False,
                   workspace: Optional[torch.Tensor] = None, stream=None) -> NVFP4Tensor:
    """Quantise a bf16 2-D CUDA tensor into `out` (see nvfp4_quantize in the header)."""
    if x.dtype != torch.bfloat16 or x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D bf16 tensor with unit column stride")
    workspace = _workspace(workspace, compute_amax, x.device)
    _check(load().nvfp4_quantize(x.data_ptr(), x.shape[0], x.shape[1], x.stride(0), int(compute_amax),
                                 SWIGLU_INTERLEAVE if interleave else 0, out.c(), _ptr(workspace),
                                 _stream(stream)), "nvfp4_quantize")
    return out


def _out2d(D: Optional[torch.Tensor]):
    if D is None:
        return None, 0
    if D.dtype != torch.bfloat16 or D.dim() != 2 or D.stride(1) != 1:
        raise ValueError("outputs are 2-D bf16 tensors with unit column stride")
    return D.data_ptr(), D.stride(0)


def gemm_nvfp4_plain(A: NVFP4Tensor, B: NVFP4Tensor, D: torch.Tensor, stream=None) -> torch.Tensor:
    p, ld = _out2d(D)
    _check(load().gemm_nvfp4_plain(A.c(), B.c(), p, ld, _stream(stream)), "gemm_nvfp4_plain")
    return D


def gemm_nvfp4_rmsnorm(A: NVFP4Tensor, B: NVFP4Tensor, w: Optional[torch.Tensor], head_dim: int,
                       n_norm_cols: int, eps: float, D: torch.Tensor, stream=None) -> torch.Tensor:
    if w is not None and (w.dtype != torch.float32 or not w.is_contiguous()):
        raise ValueError("w must be a contiguous float32 tensor")
    p, ld = _out2d(D)
    _check(load().gemm_nvfp4_rmsnorm(A.c(), B.c(), _ptr(w), head_dim, n_norm_cols, eps, p, ld, _stream(stream)),
           "gemm_nvfp4_rmsnorm")
    return D


def gemm_nvfp4_swiglu(A: NVFP4Tensor, B: NVFP4Tensor, D: Optional[torch.Tensor] = None,
                      Dq: Optional[NVFP4Tensor] = None, stream=None):
    p, ld = _out2d(D)
    dq = ctypes.pointer(Dq.c()) if Dq is not None else None
    _check(load().gemm_nvfp4_swiglu(A.c(), B.c(), p, ld, dq, _stream(stream)), "gemm_nvfp4_swiglu")
    return D, Dq


ACT_NONE, ACT_RELU = 0, 1
_OUT_KIND = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def gemm_nvfp4_pointwise(A: NVFP4Tensor, B: NVFP4Tensor, D: Optional[torch.Tensor] = None,
                         bias: Optional[torch.Tensor] = None, relu: bool = False,
                         Dq: Optional[NVFP4Tensor] = None, stream=None):
    """D = cast(act(G_A G_B acc + bias)) in D's dtype (bf16, f16 or f32) and/or Dq = NVFP4 of
    bf16 of it with Dq's static scale (see gemm_nvfp4_pointwise in the header)."""
    if bias is not None and (bias.dtype != torch.float32 or not bias.is_contiguous()):
        raise ValueError("bias must be a contiguous float32 tensor")
    if D is not None:
        if D.dtype not in _OUT_KIND or D.dim() != 2 or D.stride(1) != 1:
            raise ValueError("D must be a 2-D bf16, f16 or f32 tensor with unit column stride")
        p, ld, kind = D.data_ptr(), D.stride(0), _OUT_KIND[D.dtype]
    else:
        p, ld, kind = None, 0, 0
    dq = ctypes.pointer(Dq.c()) if Dq is not None else None
    _check(load().gemm_nvfp4_pointwise(A.c(), B.c(), _ptr(bias), ACT_RELU if relu else ACT_NONE, kind, p, ld, dq,
                                       _stream(stream)), "gemm_nvfp4_pointwise")
    return D, Dq


def gemm_nvfp4_reduce_rows_f32(A: NVFP4Tensor, B: NVFP4Tensor, dst_ptrs: torch.Tensor, rows_per_rank: int,
                               ldd: int, stream=None):
    """Add row m of G_A G_B (A B^T) (float32) into destination m // rows_per_rank at row
    m % rows_per_rank (see gemm_nvfp4_reduce_rows_f32 in the header). dst_ptrs: a device
    int64 tensor of the destinations' addresses (float32 blocks with leading dimension ldd)."""
    if dst_ptrs.dtype != torch.int64 or dst_ptrs.dim() != 1 or not dst_ptrs.is_cuda or not dst_ptrs.is_contiguous():
        raise ValueError("dst_ptrs must be a contiguous 1-D int64 tensor on the GPU")
    _check(load().gemm_nvfp4_reduce_rows_f32(A.c(), B.c(), dst_ptrs.data_ptr(), dst_ptrs.numel(), rows_per_rank, ldd,
                                             _stream(stream)), "gemm_nvfp4_reduce_rows_f32")


MXFP4_HADAMARD32 = 2


def mxfp4_quantize(x: torch.Tensor, out: NVFP4Tensor, hadamard: bool = False, interleave: bool = False,
                   stream=None) -> NVFP4Tensor:
    """MXFP4-quantise a bf16 2-D CUDA tensor (optionally after the 32-point block Hadamard
    transform, optionally with the SwiGLU gate/up row interleave) into `out` (from
    NVFP4Tensor.empty_mx); see mxfp4_quantize in the header."""
    if x.dtype != torch.bfloat16 or x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D bf16 tensor with unit column stride")
    flags = (MXFP4_HADAMARD32 if hadamard else 0) | (SWIGLU_INTERLEAVE if interleave else 0)
    _check(load().mxfp4_quantize(x.data_ptr(), x.shape[0], x.shape[1], x.stride(0), flags, out.c(),
                                 _stream(stream)), "mxfp4_quantize")
    return out


def gemm_mxfp4_rmsnorm(A: NVFP4Tensor, B: NVFP4Tensor, w: Optional[torch.Tensor], head_dim: int,
                       n_norm_cols: int, eps: float, D: torch.Tensor, stream=None) -> torch.Tensor:
    if w is not None and (w.dtype != torch.float32 or not w.is_contiguous()):
        raise ValueError("w must be a contiguous float32 tensor")
    p, ld = _out2d(D)
    _check(load().gemm_mxfp4_rmsnorm(A.c(), B.c(), _ptr(w), head_dim, n_norm_cols, eps, p, ld, _stream(stream)),
           "gemm_mxfp4_rmsnorm")
    return D


def gemm_mxfp4_swiglu(A: NVFP4Tensor, B: NVFP4Tensor, D: Optional[torch.Tensor] = None,
                      Dq: Optional[NVFP4Tensor] = None, stream=None):
    p, ld = _out2d(D)
    dq = ctypes.pointer(Dq.c()) if Dq is not None else None
    _check(load().gemm_mxfp4_swiglu(A.c(), B.c(), p, ld, dq, _stream(stream)), "gemm_mxfp4_swiglu")
    return D, Dq


def gemm_mxfp4_pointwise(A: NVFP4Tensor, B: NVFP4Tensor, D: torch.Tensor, bias: Optional[torch.Tensor] = None,
                         relu: bool = False, stream=None) -> torch.Tensor:
    if bias is not None and (bias.dtype != torch.float32 or not bias.is_contiguous()):
        raise ValueError("bias must be a contiguous float32 tensor")
    if D.dtype not in _OUT_KIND or D.dim() != 2 or D.stride(1) != 1:
        raise ValueError("D must be a 2-D bf16, f16 or f32 tensor with unit column stride")
    _check(load().gemm_mxfp4_pointwise(A.c(), B.c(), _ptr(bias), ACT_RELU if relu else ACT_NONE, _OUT_KIND[D.dtype],
                                       D.data_ptr(), D.stride(0), _stream(stream)), "gemm_mxfp4_pointwise")
    return D


def gemm_mxfp4_plain(A: NVFP4Tensor, B: NVFP4Tensor, D: torch.Tensor, stream=None) -> torch.Tensor:
    p, ld = _out2d(D)
    _check(load().gemm_mxfp4_plain(A.c(), B.c(), p, ld, _stream(stream)), "gemm_mxfp4_plain")
    return D


def rmsnorm_heads_bf16(x: torch.Tensor, w: torch.Tensor, head_dim: int, n_norm_cols: int, eps: float,
                       y: torch.Tensor, stream=None) -> torch.Tensor:
    px, ldx = _out2d(x)
    py, ldy = _out2d(y)
    _check(load().rmsnorm_heads_bf16(px, x.shape[0], ldx, w.data_ptr(), head_dim, n_norm_cols, eps, py, ldy,
                                     _stream(stream)), "rmsnorm_heads_bf16")
    return y


def swiglu_bf16(c: torch.Tensor, y: torch.Tensor, stream=None) -> torch.Tensor:
    pc, ldc = _out2d(c)
    py, ldy = _out2d(y)
    _check(load().swiglu_bf16(pc, c.shape[0], c.shape[1] // 2, ldc, py, ldy, _stream(stream)), "swiglu_bf16")
    return y


NOALLOC_MAX_VALUES = 268435456


def nvfp4_quantize_noalloc(x: torch.Tensor, out: NVFP4Tensor, interleave: bool = False, stream=None) -> NVFP4Tensor:
    """nvfp4_quantize with the per-tensor scale derived on the device, for callers that
    cannot allocate device memory: the library keeps the reduction's scratch in its own
    static device memory, so no workspace is needed (see nvfp4_quantize_noalloc in the
    header for the size limit and the rule that overlapping calls race)."""
    if x.dtype != torch.bfloat16 or x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D bf16 tensor with unit column stride")
    _check(load().nvfp4_quantize_noalloc(x.data_ptr(), x.shape[0], x.shape[1], x.stride(0),
                                         SWIGLU_INTERLEAVE if interleave else 0, out.c(), _stream(stream)),
           "nvfp4_quantize_noalloc")
    return out


def nvfp4_fake_quantize(x: torch.Tensor, y: Optional[torch.Tensor] = None, gscale: Optional[torch.Tensor] = None,
                        compute_amax: bool = True, workspace: Optional[torch.Tensor] = None, stream=None):
    """Quantise-dequantise a 2-D bf16 CUDA tensor through NVFP4 (see nvfp4_fake_quantize in
    the header). Returns (y, gscale); gscale is a 1-element float32 device tensor, written
    when compute_amax, read otherwise."""
    if x.dtype != torch.bfloat16 or x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D bf16 tensor with unit column stride")
    if y is None:
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
    py, ldy = _out2d(y)
    if gscale is None:
        if not compute_amax:
            raise ValueError("a static scale needs gscale")
        gscale = torch.empty((1,), dtype=torch.float32, device=x.device)
    workspace = _workspace(workspace, compute_amax, x.device)
    _check(load().nvfp4_fake_quantize(x.data_ptr(), x.shape[0], x.shape[1], x.stride(0), int(compute_amax),
                                      gscale.data_ptr(), py, ldy, _ptr(workspace), _stream(stream)),
           "nvfp4_fake_quantize")
    return y, gscale


class FakeQuantizeSTE(torch.autograd.Function):
    """y = nvfp4_fake_quantize(x) forward; identity backward (straight-through estimator:
    the rounding is left out of the gradient, which flows at full precision)."""

    @staticmethod
    def forward(ctx, x, gscale=None, compute_amax=True):
        y, _ = nvfp4_fake_quantize(x.contiguous(), gscale=gscale, compute_amax=compute_amax)
        return y

    @staticmethod
    def backward(ctx, grad_y):
        return grad_y, None, None


# ---- operators between the GEMMs of a layer -------------------------------------------
# Their kernels take a few microseconds at small sizes, so the checks here ask each tensor for as
# little as they can (every attribute of a tensor costs about 0.1 us).
def _same_device(*tensors: Optional[torch.Tensor]) -> int:
    """Index of the one CUDA device that all given tensors are on."""
    dev = -2
    for t in tensors:
        if t is not None:
            i = t.get_device()
            if i != dev:
                if i < 0:
                    raise ValueError("tensors must be on a CUDA device")
                if dev != -2:
                    raise ValueError("tensors must be on one device")
                dev = i
    return dev


def _call(fn, what: str, dev: int, stream, *args) -> None:
    """Call `fn` with `dev` current (the library launches on the current device), on `stream` or
    on that device's current stream."""
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)  # current_stream() would build an object: 2 us
    else:
        stream = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if torch._C._cuda_getDevice() == dev:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, stream)
    if status:
        _check(status, what)


def _stream_object(stream, device) -> torch.cuda.Stream:
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(getattr(stream, "cuda_stream", stream), device=device)


def _empty_on(stream, shape, dtype, device) -> torch.Tensor:
    """An uninitialised tensor that belongs to `stream`: its memory is neither still in use by another
    stream's work nor handed to another one before this stream's work is done."""
    with torch.cuda.stream(_stream_object(stream, device)):
        return torch.empty(shape, dtype=dtype, device=device)


ACT_SILU = 2


def _nvfp4(t: NVFP4Tensor) -> _Tensor:
    """The C form of an NVFP4 tensor whose buffers are at least as large as its size says (an MXFP4
    tensor's scales, one per 32 values, are not) and lie as its layout does."""
    rows, cols = t.rows, t.cols
    if 2 * t.codes.numel() < rows * cols or t.sf.numel() < (rows + 127) // 128 * 128 * ((cols + 63) // 64 * 4):
        raise ValueError(f"codes or scales are too small for an NVFP4 tensor of {rows} x {cols}")
    if not (t.codes.is_contiguous() and t.sf.is_contiguous()):
        raise ValueError("codes and scales must be contiguous")
    if t.gscale.dtype is not torch.float32:
        raise ValueError("gscale must be float32")
    return t.c()


def _pitch(stride, rows: int, cols: int) -> int:
    """Row pitch from a 2-D tensor's strides. One row has no pitch, and torch may report any: it gets
    that of a buffer of its own."""
    return stride[0] if rows > 1 else (cols + 7) // 8 * 8


def gemv_nvfp4(x: torch.Tensor, B: NVFP4Tensor, D: torch.Tensor, bias: Optional[torch.Tensor] = None,
               silu: bool = False, stream=None) -> torch.Tensor:
    """D = cast(f(x) (G B)^T + bias) for a few rows x (M x K, bf16 or f16) and an NVFP4 weight B
    (N x K); f is the identity or SiLU; D (M x N) is bf16, f16 or f32 (see gemv_nvfp4 in the
    header). For serving: D takes no part in a graph."""
    x_dtype, sx, D_dtype, sD = x.dtype, x.stride(), D.dtype, D.stride()
    if len(sx) != 2 or sx[1] != 1 or (x_dtype is not torch.bfloat16 and x_dtype is not torch.float16):
        raise ValueError("x must be a 2-D bf16 or f16 tensor with unit column stride")
    M, K = x.shape
    N = B.rows
    if D_dtype not in _OUT_KIND or len(sD) != 2 or (sD[1] != 1 and N > 1):
        raise ValueError("D must be a 2-D bf16, f16 or f32 tensor with unit column stride")
    if K != B.cols or D.shape != (M, N):
        raise ValueError(f"x is {M} x {K}, B {N} x {B.cols} and D {tuple(D.shape)}")
    if bias is not None and (bias.dtype is not torch.float32 or bias.shape != (N,) or not bias.is_contiguous()):
        raise ValueError("bias must be a contiguous float32 tensor with one value per row of B")
    dev = _same_device(x, D, B.codes, B.sf, B.gscale, bias)
    _call((_lib or load()).gemv_nvfp4, "gemv_nvfp4", dev, stream, x.data_ptr(), _OUT_KIND[x_dtype], M,
          sx[0] if M > 1 else _pitch(sx, M, K), ACT_SILU if silu else ACT_NONE, _nvfp4(B),
          None if bias is None else bias.data_ptr(), _OUT_KIND[D_dtype], D.data_ptr(),
          sD[0] if M > 1 else _pitch(sD, M, N))
    return D


_NORMS = {None: 0, "layer": 1, "rms": 2}
# nvfp4_norm_inputs and nvfp4_norm_grads of the header, packed in one step (a ctypes structure of as
# many fields takes 3 us to fill)
_NORM_INPUTS = struct.Struct("@3qP4i2f" + "Pq" * 5 + "2P")
_NORM_GRADS = struct.Struct("@" + "Pq" * 7 + "2P")


def _matrix(t: torch.Tensor, name: str, shape, dtype):
    """Pointer and row pitch of a 2-D tensor of the given shape and type."""
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name} must be a {shape[0]} x {shape[1]} {dtype} tensor with unit column stride")
    pitch, one = t.stride()
    if one != 1:
        raise ValueError(f"{name} must be a {shape[0]} x {shape[1]} {dtype} tensor with unit column stride")
    return t.data_ptr(), pitch if shape[0] > 1 else _pitch((pitch,), 1, shape[1])


_NONE = (0, 0)  # the pointer and pitch of a matrix that is not given


def _vector(t: torch.Tensor, name: str, cols: int):
    if t.dtype is not torch.float32 or t.shape != (cols,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor of {cols} values")
    return t.data_ptr()


def _norm_inputs(x, y, gate, scale, shift, w, w_post, norm, post_norm, residual_scale, eps, offsets, batches):
    """The inputs checked and packed, and the modulation tensors' shape."""
    x_dtype, sx, x_shape = x.dtype, x.stride(), x.shape
    if len(sx) != 2 or sx[1] != 1 or (x_dtype is not torch.bfloat16 and x_dtype is not torch.float32):
        raise ValueError("the stream must be a 2-D bf16 or float32 tensor with unit column stride")
    if norm not in _NORMS:
        raise ValueError('norm must be "layer", "rms" or None')
    rows, cols = x_shape
    mod = gate if gate is not None else scale if scale is not None else shift
    if offsets is not None:
        if offsets.dtype is not torch.int32 or offsets.dim() != 1 or offsets.shape[0] < 2 or not offsets.is_contiguous():
            raise ValueError("offsets must be a contiguous 1-D int32 tensor of batches + 1 values")
        n = offsets.shape[0] - 1
        if batches is not None and batches != n:
            raise ValueError("batches does not agree with offsets")
        batches = n
    elif batches is None:
        batches = mod.shape[0] if mod is not None else 1
    mod_dtype = mod.dtype if mod is not None else torch.float32
    if mod_dtype is not torch.bfloat16 and mod_dtype is not torch.float32:
        raise ValueError("gate, scale and shift must be bf16 or float32")
    shape = (batches, cols)
    return _NORM_INPUTS.pack(
        rows, cols, batches, 0 if offsets is None else offsets.data_ptr(), _OUT_KIND[x_dtype], _OUT_KIND[mod_dtype],
        _NORMS[norm], post_norm, residual_scale, eps, x.data_ptr(), sx[0] if rows > 1 else _pitch(sx, rows, cols),
        *(_NONE if y is None else _matrix(y, "y", x_shape, torch.bfloat16)),
        *(_NONE if gate is None else _matrix(gate, "gate", shape, mod_dtype)),
        *(_NONE if scale is None else _matrix(scale, "scale", shape, mod_dtype)),
        *(_NONE if shift is None else _matrix(shift, "shift", shape, mod_dtype)),
        0 if w_post is None else _vector(w_post, "w_post", cols), 0 if w is None else _vector(w, "w", cols)), shape


def _stats(stats, rows):
    if stats.dtype is not torch.float32 or stats.shape != (rows, 4) or not stats.is_contiguous():
        raise ValueError("stats must be a contiguous rows x 4 float32 tensor")


def residual_norm(x: torch.Tensor, h: Optional[torch.Tensor] = None, hq: Optional[NVFP4Tensor] = None, *,
                  y: Optional[torch.Tensor] = None, x_out: Optional[torch.Tensor] = None,
                  gate: Optional[torch.Tensor] = None, post_norm: bool = False,
                  w_post: Optional[torch.Tensor] = None, residual_scale: float = 1.0, norm: Optional[str] = "layer",
                  w: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                  shift: Optional[torch.Tensor] = None, eps: float = 1e-6,
                  offsets: Optional[torch.Tensor] = None, batches: Optional[int] = None,
                  stats: Optional[torch.Tensor] = None, stream=None):
    """x_out = residual_scale x + gate y~ (y~ = y or its RMSNorm), and the norm of x_out, modulated,
    into h (bf16) and / or hq (NVFP4 with hq's static scale); see residual_norm in the header.

    x, x_out: rows x cols, bf16 or float32; y: bf16. gate, scale, shift: batches x cols, bf16 or
    float32 alike, possibly slices of one tensor. w, w_post: cols float32. offsets: batches + 1
    int32 row offsets on the device (None: sequences of equal length); rows without a sequence are
    left as they are. stats: rows x 4 float32, written for residual_norm_backward. Outputs that are
    None are not written. Returns (x_out, h, hq), which take no part in a graph (ResidualNorm's do)."""
    dev = _same_device(x, h, y, x_out, gate, w_post, w, scale, shift, offsets, stats)
    if hq is not None:
        _same_device(x, hq.codes, hq.sf, hq.gscale)
    a, _ = _norm_inputs(x, y, gate, scale, shift, w, w_post, norm, post_norm, residual_scale, eps, offsets, batches)
    shape = x.shape
    if stats is not None:
        _stats(stats, shape[0])
    _call((_lib or load()).residual_norm, "residual_norm", dev, stream, a,
          *(_NONE if x_out is None else _matrix(x_out, "x_out", shape, x.dtype)),
          *(_NONE if h is None else _matrix(h, "h", shape, torch.bfloat16)), ctypes.pointer(_nvfp4(hq)) if hq is not None else None,
          None if stats is None else stats.data_ptr())
    return x_out, h, hq


def residual_norm_workspace_bytes(rows: int, cols: int, batches: int) -> int:
    return int((_lib or load()).residual_norm_workspace_bytes(rows, cols, batches))


def residual_norm_backward(x_out: torch.Tensor, stats: torch.Tensor, *, dx_out: Optional[torch.Tensor] = None,
                           dh: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                           gate: Optional[torch.Tensor] = None, post_norm: bool = False,
                           w_post: Optional[torch.Tensor] = None, residual_scale: float = 1.0,
                           norm: Optional[str] = "layer", w: Optional[torch.Tensor] = None,
                           scale: Optional[torch.Tensor] = None, eps: float = 1e-6,
                           offsets: Optional[torch.Tensor] = None, batches: Optional[int] = None,
                           dx: Optional[torch.Tensor] = None, dy: Optional[torch.Tensor] = None,
                           dgate: Optional[torch.Tensor] = None, dscale: Optional[torch.Tensor] = None,
                           dshift: Optional[torch.Tensor] = None, dw: Optional[torch.Tensor] = None,
                           dw_post: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                           stream=None) -> None:
    """Gradient of residual_norm from those of its outputs (dx_out, dh; None: 0), into whichever of
    dx, dy (as x, y), dgate, dscale, dshift (batches x cols float32), dw and dw_post (cols float32)
    are given; they are overwritten. x_out is the stream that the forward call stored, stats what it
    wrote there (see residual_norm_backward in the header)."""
    dev = _same_device(x_out, stats, dx_out, dh, y, gate, w_post, w, scale, offsets, dx, dy, dgate, dscale, dshift,
                       dw, dw_post, workspace)
    seq = dgate if dgate is not None else dscale if dscale is not None else dshift
    if batches is None and offsets is None and gate is None and scale is None and seq is not None:
        batches = seq.shape[0]
    a, shape = _norm_inputs(x_out, y, gate, scale, None, w, w_post, norm, post_norm, residual_scale, eps, offsets, batches)
    full, dtype, bf16, f32 = x_out.shape, x_out.dtype, torch.bfloat16, torch.float32
    rows, cols = full
    _stats(stats, rows)
    g = _NORM_GRADS.pack(*(_NONE if dx_out is None else _matrix(dx_out, "dx_out", full, dtype)),
                         *(_NONE if dh is None else _matrix(dh, "dh", full, bf16)),
                         *(_NONE if dx is None else _matrix(dx, "dx", full, dtype)),
                         *(_NONE if dy is None else _matrix(dy, "dy", full, bf16)),
                         *(_NONE if dgate is None else _matrix(dgate, "dgate", shape, f32)),
                         *(_NONE if dscale is None else _matrix(dscale, "dscale", shape, f32)),
                         *(_NONE if dshift is None else _matrix(dshift, "dshift", shape, f32)),
                         0 if dw is None else _vector(dw, "dw", cols),
                         0 if dw_post is None else _vector(dw_post, "dw_post", cols))
    if seq is not None or dw is not None or dw_post is not None:
        need = residual_norm_workspace_bytes(rows, cols, shape[0])
        if workspace is None:
            # (new_empty takes half of torch.empty's 2 us)
            workspace = x_out.new_empty((need,), dtype=torch.uint8) if stream is None else (
                _empty_on(stream, (need,), torch.uint8, x_out.device))
        else:
            _check_workspace(workspace, need)
    _call((_lib or load()).residual_norm_backward, "residual_norm_backward", dev, stream, a, stats.data_ptr(), g,
          None if workspace is None else workspace.data_ptr())


def _aligned(t: torch.Tensor) -> torch.Tensor:
    """`t`, copied unless each of its rows can be read 16 bytes at a time. (A copy by contiguous()
    would return a contiguous view as it is, wherever it starts.)"""
    size = t.element_size()
    if t.stride(-1) == 1 and t.data_ptr() % 16 == 0 and all(
            n == 1 or s * size % 16 == 0 for n, s in zip(t.shape[:-1], t.stride())):
        return t
    return t.clone(memory_format=torch.contiguous_format)


def _rows_of_16_bytes(t: torch.Tensor) -> torch.Tensor:
    """The same for a matrix whose rows may not overlap either (a broadcast gradient)."""
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        return t.clone(memory_format=torch.contiguous_format)
    return _aligned(t)


class ResidualNorm(torch.autograd.Function):
    """residual_norm with its gradient: apply(x, y, gate, scale, shift, w, w_post, norm, post_norm,
    residual_scale, eps, offsets) returns (x_out, h); h alone without a branch (y None), x_out alone
    with norm None. Rows without a sequence are 0 in the outputs and in the gradients. Parameters'
    gradients are summed in float32 and returned in the parameter's type. Inputs and gradients that the
    kernels cannot read 16 bytes at a time are copied first."""

    @staticmethod
    def forward(ctx, x, y=None, gate=None, scale=None, shift=None, w=None, w_post=None, norm="layer",
                post_norm=False, residual_scale=1.0, eps=1e-6, offsets=None):
        if y is None and norm is None:
            raise ValueError("without a branch and a norm there is nothing to compute")
        x, y, gate, scale, shift = (None if t is None else _rows_of_16_bytes(t) for t in (x, y, gate, scale, shift))
        w, w_post = (None if t is None else _aligned(t) for t in (w, w_post))
        make = torch.empty if offsets is None else torch.zeros
        x_out = make(x.shape, dtype=x.dtype, device=x.device) if y is not None else None
        h = make(x.shape, dtype=torch.bfloat16, device=x.device) if norm is not None else None
        stats = make((x.shape[0], 4), dtype=torch.float32, device=x.device)
        mods = [m for m in (gate, scale, shift) if m is not None]
        batches = mods[0].shape[0] if mods and offsets is None else None
        residual_norm(x, h, y=y, x_out=x_out, gate=gate, post_norm=post_norm, w_post=w_post,
                      residual_scale=residual_scale, norm=norm, w=w, scale=scale, shift=shift, eps=eps,
                      offsets=offsets, batches=batches, stats=stats)
        ctx.save_for_backward(x_out if y is not None else x, y, gate, scale, shift, w, w_post, offsets, stats)
        ctx.args = (norm, post_norm, residual_scale, eps, batches)
        ctx.set_materialize_grads(False)
        if y is None:
            return h
        return (x_out, h) if norm is not None else x_out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, *grads):
        x_out, y, gate, scale, shift, w, w_post, offsets, stats = ctx.saved_tensors
        norm, post_norm, residual_scale, eps, batches = ctx.args
        if y is None:
            dx_out, dh = None, grads[0]
        else:
            dx_out, dh = grads if norm is not None else (grads[0], None)
        if dx_out is None and dh is None:
            return (None,) * 12
        dx_out = None if dx_out is None else _rows_of_16_bytes(dx_out)
        dh = None if dh is None else _rows_of_16_bytes(dh)
        need = ctx.needs_input_grad + (False,) * 12  # arguments that were left out need none
        make = torch.empty_like if offsets is None else torch.zeros_like

        def like(i, t):
            return make(t, memory_format=torch.contiguous_format) if need[i] and t is not None else None

        def sums(i, t):
            return torch.empty(t.shape, dtype=torch.float32, device=t.device) if need[i] and t is not None else None

        dx, dy = like(0, x_out), like(1, y)
        dgate, dscale, dshift = sums(2, gate), sums(3, scale), sums(4, shift)
        dw, dw_post = sums(5, w), sums(6, w_post)
        if any(t is not None for t in (dx, dy, dgate, dscale, dshift, dw, dw_post)):
            residual_norm_backward(x_out, stats, dx_out=dx_out, dh=dh, y=y, gate=gate, post_norm=post_norm,
                                   w_post=w_post, residual_scale=residual_scale, norm=norm, w=w, scale=scale, eps=eps,
                                   offsets=offsets, batches=batches, dx=dx, dy=dy, dgate=dgate, dscale=dscale,
                                   dshift=dshift, dw=dw, dw_post=dw_post)

        def cast(d, t):
            return None if d is None else d.to(t.dtype)

        return (dx, dy, cast(dgate, gate), cast(dscale, scale), cast(dshift, shift), dw, dw_post,
                None, None, None, None, None)


def rope_frequencies(pairs, theta: float = 10000.0, device="cuda") -> torch.Tensor:
    """Frequencies of rope_axes: for an axis of n pairs, theta^(-j / n), j = 0 .. n - 1 (float64)."""
    return torch.cat([theta ** (-torch.arange(n, dtype=torch.float64) / n) for n in pairs]).to(device)


@functools.lru_cache(maxsize=256)
def _axis_pairs(pairs: tuple):
    return (ctypes.c_int32 * len(pairs))(*pairs), len(pairs), sum(pairs)


def rope_axes(x: torch.Tensor, positions: torch.Tensor, freqs: torch.Tensor, pairs, y: Optional[torch.Tensor] = None,
              interleaved: bool = True, inverse: bool = False, stream=None) -> torch.Tensor:
    """Rotary positions on heads x (rows x heads x head_dim; bf16, f16 or f32) into y, which may be
    x itself (None: a new contiguous tensor, allocated on `stream`). positions: rows x axes, int32 or float32; pairs: how
    many pairs each axis turns; freqs: one float64 per pair (rope_frequencies). inverse: the
    opposite rotation, which is also the gradient (see rope_axes in the header). A new result carries
    x's gradient, as RopeAxes' does; a given y is written to and takes no part in a graph."""
    if y is None and x.requires_grad and torch.is_grad_enabled():
        if stream is None:
            return RopeAxes.apply(x, positions, freqs, pairs, interleaved, inverse)
        with torch.cuda.stream(_stream_object(stream, x.device)):
            return RopeAxes.apply(x, positions, freqs, pairs, interleaved, inverse)
    dtype, sx, shape = x.dtype, x.stride(), x.shape
    if len(sx) != 3 or sx[2] != 1 or dtype not in _OUT_KIND:
        raise ValueError("x must be a rows x heads x head_dim tensor (bf16, f16 or f32) with unit last stride")
    if y is None:
        y = torch.empty_like(x, memory_format=torch.contiguous_format) if stream is None else (
            _empty_on(stream, shape, dtype, x.device))
    sy = y.stride()
    if y.shape != shape or y.dtype is not dtype or sy[2] != 1:
        raise ValueError("y must have x's shape and type and unit last stride")
    rows, heads, head_dim = shape
    c_pairs, axes, n = _axis_pairs(tuple(pairs))
    p_dtype, sp = positions.dtype, positions.stride()
    if positions.shape != (rows, axes) or (p_dtype is not torch.int32 and p_dtype is not torch.float32) or (
            axes > 1 and sp[1] != 1):
        raise ValueError("positions must be rows x axes int32 or float32 with unit column stride")
    if freqs.dtype is not torch.float64 or freqs.shape != (n,) or not freqs.is_contiguous():
        raise ValueError("freqs must be a contiguous float64 tensor with one value per pair")
    dev = _same_device(x, y, positions, freqs)
    _call((_lib or load()).rope_axes, "rope_axes", dev, stream, x.data_ptr(), _OUT_KIND[dtype], rows, heads, head_dim,
          sx[0], sx[1], positions.data_ptr(), p_dtype is torch.float32, sp[0] if rows > 1 else axes, axes, c_pairs,
          freqs.data_ptr(), interleaved, inverse, y.data_ptr(), sy[0], sy[1])
    return y


class RopeAxes(torch.autograd.Function):
    """rope_axes with its gradient (the opposite rotation): apply(x, positions, freqs, pairs,
    interleaved, inverse). Positions and frequencies get none. x and its gradient are copied first where the
    kernel cannot read them 16 bytes at a time."""

    @staticmethod
    def forward(ctx, x, positions, freqs, pairs, interleaved=True, inverse=False):
        ctx.save_for_backward(positions, freqs)
        ctx.args = (tuple(pairs), interleaved, inverse)
        return rope_axes(_aligned(x), positions, freqs, pairs, interleaved=interleaved, inverse=inverse)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        positions, freqs = ctx.saved_tensors
        pairs, interleaved, inverse = ctx.args
        dx = rope_axes(_aligned(dy), positions, freqs, pairs, interleaved=interleaved, inverse=not inverse)
        return dx, None, None, None, None, None


def read_device_status(stream=None) -> int:
    return int(load().nvfp4_read_device_status(_stream(stream)))


def signal_barrier(signal_ptrs: torch.Tensor, rank: int, epoch: int, limit_ns: int = 10_000_000_000,
                   stream=None) -> None:
    """Barrier over peer-mapped signal words: signal_ptrs is a device int64 tensor of the
    world's signal-array addresses (see nvfp4_signal_barrier). A rank that does not arrive
    within limit_ns ends this rank's wait with NVFP4_ERR_DEVICE_TIMEOUT in the device status
    word (read_device_status) instead of holding the GPU."""
    if signal_ptrs.dtype != torch.int64 or not signal_ptrs.is_cuda:
        raise RuntimeError("signal_ptrs must be a CUDA int64 tensor of addresses")
    _check(load().nvfp4_signal_barrier(signal_ptrs.data_ptr(), signal_ptrs.numel(), rank, epoch & 0xFFFFFFFF,
                                       limit_ns, _stream(stream)), "nvfp4_signal_barrier")


def selftest_bounded_wait(limit_ns: int, stream=None) -> None:
    _check(load().nvfp4_selftest_bounded_wait(limit_ns, _stream(stream)), "nvfp4_selftest_bounded_wait")


def launch_count() -> int:
    return int(load().nvfp4_launch_count())
