"""Python binding of libmx_gb300.so (the C ABI in include/mx.h).

Argument marshalling only: every step of quantization and matrix multiply runs
in the library's CUDA kernels.  PyTorch supplies device memory and the current
stream.  There is no fallback: if the shared library is missing or fails to
load, every call raises.

    from block_scaled_quantized_mx_gb300 import mx_quantize, mx_gemm, gemm_f16
    a = mx_quantize(A_fp32, E4M3)                      # A: M x K, K contiguous
    b = mx_quantize(B_fp32, E4M3, k_strided=True)      # B: K x N row-major
    C = mx_gemm(a, b, out_dtype=torch.bfloat16)        # C = A @ B
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass

import torch

from . import _build

E4M3 = 1
E2M1 = 2
E5M2 = 3
INT8 = 4
INT4 = 5
INT2 = 6
DT_F32, DT_BF16, DT_F16 = 0, 1, 2
SRC_K_CONTIGUOUS, SRC_K_STRIDED = 0, 1
ACT_NONE, ACT_GELU, ACT_GELU_TANH = 0, 1, 2

STATUS = {0: "MX_OK", 1: "MX_ERR_INVALID_ARG", 2: "MX_ERR_SHAPE",
          3: "MX_ERR_ALIGN", 4: "MX_ERR_UNSUPPORTED", 5: "MX_ERR_CUDA",
          6: "MX_ERR_TIMEOUT"}

EXPORTS = ("mx_data_bytes", "mx_scale_bytes", "mx_quantize", "mx_gemm",
           "gemm_f16", "mx_gemm_fused", "mx_gemm_fused_quantize",
           "gemm_f16_fused", "gemm_dequant", "gemm_dequant_splitk",
           "gemm_dequant_workspace_bytes", "flash_attention",
           "flash_attention_workspace_bytes", "flash_attention_splitkv",
           "mx_gemm_workspace_bytes",
           "mx_gemm_splitk",
           "gemm_f16_workspace_bytes", "gemm_f16_splitk",
           "mx_gemm_splitk_noalloc", "mx_last_error",
           "mx_selftest_wait_timeout", "mx_scales_to_rowmajor",
           "mx_status_string", "mx_version", "mx_set_tile_width",
           "mx_kv_extend", "mx_kv_truncate", "mx_kv_append",
           "mx_kv_attention_workspace_bytes", "mx_kv_attention")


class MXError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__("%s failed: %s" % (what, STATUS.get(status, status)))
        self.status = status


class CMXTensor(ctypes.Structure):
    """Mirror of struct mx_tensor."""
    _fields_ = [("data", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("fmt", ctypes.c_int32), ("outer", ctypes.c_int64),
                ("K", ctypes.c_int64)]


class CEpilogue(ctypes.Structure):
    """Mirror of struct mx_epilogue."""
    _fields_ = [("bias", ctypes.c_void_p), ("act", ctypes.c_int32)]


class CKVCache(ctypes.Structure):
    """Mirror of struct mx_kv_cache."""
    _fields_ = [("k_data", ctypes.c_void_p), ("v_data", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("fmt", ctypes.c_int32), ("page", ctypes.c_int32),
                ("pages", ctypes.c_int64), ("heads", ctypes.c_int64),
                ("d", ctypes.c_int64)]


_lib = None


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the CUDA sources for sm_103a into the in-tree shared library."""
    return _build.build(force=force, verbose=verbose)


def lib_path() -> str:
    return _build.LIB_PATH


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_build.LIB_PATH):
        raise RuntimeError("%s is not built: call "
                           "block_scaled_quantized_mx_gb300.build() first"
                           % _build.LIB_PATH)
    L = ctypes.CDLL(_build.LIB_PATH)
    i32, i64, p, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, \
        ctypes.c_size_t
    pt = ctypes.POINTER(CMXTensor)
    L.mx_data_bytes.restype = sz
    L.mx_data_bytes.argtypes = [i32, i64, i64]
    L.mx_scale_bytes.restype = sz
    L.mx_scale_bytes.argtypes = [i64, i64]
    L.mx_quantize.restype = i32
    L.mx_quantize.argtypes = [p, i64, i32, pt, p]
    L.mx_gemm.restype = i32
    L.mx_gemm.argtypes = [pt, pt, p, i32, i64, p]
    L.gemm_f16.restype = i32
    L.gemm_f16.argtypes = [p, p, p, i32, i64, i64, i64, i64, i64, i64, p]
    pe = ctypes.POINTER(CEpilogue)
    L.mx_gemm_fused.restype = i32
    L.mx_gemm_fused.argtypes = [pt, pt, pe, p, i32, i64, p]
    L.mx_gemm_fused_quantize.restype = i32
    L.mx_gemm_fused_quantize.argtypes = [pt, pt, pe, pt, p]
    L.gemm_f16_fused.restype = i32
    L.gemm_f16_fused.argtypes = [p, p, pe, p, i32, i64, i64, i64, i64, i64,
                                 i64, p]
    L.gemm_dequant.restype = i32
    L.gemm_dequant.argtypes = [p, i32, i64, i64, pt, pe, p, i32, i64, p]
    L.gemm_dequant_splitk.restype = i32
    L.gemm_dequant_splitk.argtypes = [p, i32, i64, i64, pt, pe, p, i32, i64, p,
                                      sz, p]
    L.gemm_dequant_workspace_bytes.restype = sz
    L.gemm_dequant_workspace_bytes.argtypes = [i64, i64, i64]
    L.flash_attention.restype = i32
    L.flash_attention.argtypes = [p, p, p, p, i32, i32, i64, i64, i64, i64,
                                  ctypes.c_float, p]
    L.flash_attention_workspace_bytes.restype = sz
    L.flash_attention_workspace_bytes.argtypes = [i64, i64, i64, i64]
    L.flash_attention_splitkv.restype = i32
    L.flash_attention_splitkv.argtypes = [p, p, p, p, i32, i32, i64, i64, i64,
                                          i64, ctypes.c_float, p, sz, p]
    L.mx_gemm_workspace_bytes.restype = sz
    L.mx_gemm_workspace_bytes.argtypes = [i32, i64, i64, i64]
    L.mx_gemm_splitk.restype = i32
    L.mx_gemm_splitk.argtypes = [pt, pt, p, i32, i64, p, sz, p]
    L.gemm_f16_workspace_bytes.restype = sz
    L.gemm_f16_workspace_bytes.argtypes = [i64, i64, i64]
    L.gemm_f16_splitk.restype = i32
    L.gemm_f16_splitk.argtypes = [p, p, p, i32, i64, i64, i64, i64, i64, i64,
                                  p, sz, p]
    L.mx_gemm_splitk_noalloc.restype = i32
    L.mx_gemm_splitk_noalloc.argtypes = [pt, pt, p, i32, i64, p]
    L.mx_last_error.restype = i32
    L.mx_last_error.argtypes = [p]
    L.mx_selftest_wait_timeout.restype = i32
    L.mx_selftest_wait_timeout.argtypes = [i64, p]
    L.mx_scales_to_rowmajor.restype = i32
    L.mx_scales_to_rowmajor.argtypes = [p, p, i64, i64]
    L.mx_status_string.restype = ctypes.c_char_p
    L.mx_status_string.argtypes = [i32]
    L.mx_version.restype = i32
    L.mx_version.argtypes = []
    L.mx_set_tile_width.restype = i32
    L.mx_set_tile_width.argtypes = [i32]
    pc = ctypes.POINTER(CKVCache)
    L.mx_kv_extend.restype = i32
    L.mx_kv_extend.argtypes = [p, p, i64, p, i64, i64, p, i64, p, i32, p, p, p,
                               i64, p, p]
    L.mx_kv_truncate.restype = i32
    L.mx_kv_truncate.argtypes = [p, p, i64, p, i64, i64, p, i64, p, i32, p, p,
                                 p]
    L.mx_kv_append.restype = i32
    L.mx_kv_append.argtypes = [pc, p, p, i32, i64, i64, i64, i64, i64, p, p]
    L.mx_kv_attention_workspace_bytes.restype = sz
    L.mx_kv_attention_workspace_bytes.argtypes = [i64, i64, i64, i64]
    L.mx_kv_attention.restype = i32
    L.mx_kv_attention.argtypes = [p, i32, i64, i64, i64, i64, pc, p, i64, i64,
                                  p, p, i64, i64, p, i32, i64, i64, i32, i64,
                                  ctypes.c_float, p, sz, p]
    _lib = L
    return L


def _stream(stream) -> int:
    if stream is None:
        # the handle alone: building a Stream object for it takes 3 us
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, what: str):
    if status != 0:
        raise MXError(status, what)


@dataclass
class MXTensor:
    """An MX tensor: data plane and scale plane (device uint8 tensors) of an
    outer x K matrix, K being the contraction axis."""
    data: torch.Tensor
    scales: torch.Tensor
    fmt: int
    outer: int
    K: int

    def c(self) -> CMXTensor:
        return CMXTensor(self.data.data_ptr() if self.data.numel() else None,
                         self.scales.data_ptr() if self.scales.numel() else None,
                         self.fmt, self.outer, self.K)


@functools.lru_cache(maxsize=1024)
def data_bytes(fmt: int, outer: int, K: int) -> int:
    return int(lib().mx_data_bytes(fmt, outer, K))


@functools.lru_cache(maxsize=1024)
def scale_bytes(outer: int, K: int) -> int:
    return int(lib().mx_scale_bytes(outer, K))


def empty_mx(fmt: int, outer: int, K: int, device="cuda") -> MXTensor:
    nd = data_bytes(fmt, outer, K)
    ns = scale_bytes(outer, K)
    return MXTensor(torch.empty(nd, dtype=torch.uint8, device=device),
                    torch.empty(ns, dtype=torch.uint8, device=device),
                    fmt, outer, K)


def _check_mx(t: MXTensor, name: str, fmt=None, outer=None, K=None):
    """An MX tensor's planes are contiguous buffers holding at least the
    bytes the library reads or writes for its format and shape (the C ABI
    receives bare pointers and cannot check their extent)."""
    if ((fmt is not None and t.fmt != fmt) or
            (outer is not None and t.outer != outer) or
            (K is not None and t.K != K)):
        raise ValueError(f"{name} must be format {fmt}, {outer} x {K}")
    for plane, need in ((t.data, data_bytes(t.fmt, t.outer, t.K)),
                        (t.scales, scale_bytes(t.outer, t.K))):
        if not plane.is_contiguous():
            raise ValueError(f"{name}: planes must be contiguous")
        if plane.numel() * plane.element_size() < need:
            raise ValueError(f"{name}: a plane holds fewer than the {need} "
                             "bytes its format and shape need")


def _check_out(out: torch.Tensor, rows: int, cols: int, dtype):
    """A caller-supplied output matrix: of the requested dtype, on the GPU,
    rows x cols with a unit inner stride (its row stride becomes ldc)."""
    if out.dtype != dtype or not out.is_cuda:
        raise ValueError(f"out must be a {dtype} CUDA tensor")
    if out.dim() != 2 or tuple(out.shape) != (rows, cols):
        raise ValueError(f"out must be {rows} x {cols}")
    if cols > 1 and out.stride(1) != 1:
        raise ValueError("out must have a unit inner stride")


def _out_code(dtype, allowed) -> int:
    """The C ABI's code for an output dtype among those a call supports."""
    if dtype not in allowed:
        raise ValueError("out_dtype must be one of %s, not %s"
                         % (", ".join(str(a) for a in allowed), dtype))
    return {torch.float32: DT_F32, torch.bfloat16: DT_BF16,
            torch.float16: DT_F16}[dtype]


def _nbytes(t: torch.Tensor | None) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def mx_quantize(src: torch.Tensor, fmt: int, k_strided: bool = False,
                out: MXTensor | None = None, stream=None) -> MXTensor:
    """Quantize a 2-D fp32 CUDA tensor.  ``k_strided=False``: src is
    outer x K; ``k_strided=True``: src is K x outer (e.g. a row-major K x N
    B operand).  The row stride may exceed the width."""
    if src.dtype != torch.float32 or src.dim() != 2 or not src.is_cuda:
        raise ValueError("src must be a 2-D float32 CUDA tensor")
    if src.stride(1) != 1:
        raise ValueError("src must have a unit inner stride")
    if k_strided:
        K, outer = src.shape
    else:
        outer, K = src.shape
    if out is None:
        out = empty_mx(fmt, outer, K, src.device)
    _check_mx(out, "out", fmt, outer, K)
    ct = out.c()
    _check(lib().mx_quantize(src.data_ptr(), src.stride(0),
                             SRC_K_STRIDED if k_strided else SRC_K_CONTIGUOUS,
                             ctypes.byref(ct), _stream(stream)), "mx_quantize")
    return out


def mx_gemm_workspace_bytes(fmt: int, M: int, N: int, K: int) -> int:
    return int(lib().mx_gemm_workspace_bytes(fmt, M, N, K))


def gemm_f16_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib().gemm_f16_workspace_bytes(M, N, K))


def mx_gemm(A: MXTensor, B: MXTensor, out_dtype=torch.bfloat16,
            out: torch.Tensor | None = None, stream=None,
            workspace: torch.Tensor | None = None) -> torch.Tensor:
    """C = A * B for MX tensors A (M x K) and B (quantized from K x N); the
    two may hold different element formats.  With a workspace (a CUDA tensor of at least mx_gemm_workspace_bytes()
    bytes) the K-split entry point is used."""
    dt = _out_code(out_dtype, (torch.float32, torch.bfloat16))
    _check_mx(A, "A")
    _check_mx(B, "B")
    if out is None:
        out = torch.empty((A.outer, B.outer), dtype=out_dtype,
                          device=A.data.device)
    _check_out(out, A.outer, B.outer, out_dtype)
    ca, cb = A.c(), B.c()
    cptr = out.data_ptr() if out.numel() else None
    ldc = out.stride(0)
    if workspace is None:
        _check(lib().mx_gemm(ctypes.byref(ca), ctypes.byref(cb), cptr, dt, ldc,
                             _stream(stream)), "mx_gemm")
    else:
        _check(lib().mx_gemm_splitk(
            ctypes.byref(ca), ctypes.byref(cb), cptr, dt, ldc,
            workspace.data_ptr() if workspace.numel() else None,
            _nbytes(workspace), _stream(stream)),
            "mx_gemm_splitk")
    return out


def gemm_f16(A: torch.Tensor, B: torch.Tensor, out: torch.Tensor | None = None,
             stream=None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """C (fp32) = A * B for row-major fp16 or bf16 CUDA tensors."""
    if A.dtype != B.dtype or A.dtype not in (torch.float16, torch.bfloat16):
        raise ValueError("A and B must both be fp16 or both bf16")
    M, K = A.shape
    K2, N = B.shape
    if K != K2:
        raise ValueError("inner dimensions differ")
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=A.device)
    _check_out(out, M, N, torch.float32)
    dt = DT_F16 if A.dtype == torch.float16 else DT_BF16
    args = (A.data_ptr() if A.numel() else None,
            B.data_ptr() if B.numel() else None,
            out.data_ptr() if out.numel() else None, dt, M, N, K,
            A.stride(0), B.stride(0), out.stride(0))
    if workspace is None:
        _check(lib().gemm_f16(*args, _stream(stream)), "gemm_f16")
    else:
        _check(lib().gemm_f16_splitk(
            *args, workspace.data_ptr() if workspace.numel() else None,
            _nbytes(workspace), _stream(stream)),
            "gemm_f16_splitk")
    return out


def _epilogue(bias, act) -> CEpilogue:
    if bias is not None:
        if (bias.dtype != torch.float32 or bias.dim() != 1 or not bias.is_cuda
                or not bias.is_contiguous()):
            raise ValueError("bias must be a contiguous 1-D float32 CUDA tensor")
    return CEpilogue(bias.data_ptr() if bias is not None and bias.numel() else
                     None, int(act))


def _check_bias(bias, N):
    if bias is not None and bias.numel() != N:
        raise ValueError("bias must hold N values")


def mx_gemm_fused(A: MXTensor, B: MXTensor, bias: torch.Tensor | None = None,
                  act: int = ACT_NONE, out_dtype=torch.bfloat16,
                  out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """C = act(A * B + bias) with the bias and activation applied to the
    fp32 accumulator inside the GEMM epilogue."""
    _check_bias(bias, B.outer)
    dt = _out_code(out_dtype, (torch.float32, torch.bfloat16))
    _check_mx(A, "A")
    _check_mx(B, "B")
    if out is None:
        out = torch.empty((A.outer, B.outer), dtype=out_dtype,
                          device=A.data.device)
    _check_out(out, A.outer, B.outer, out_dtype)
    ca, cb, ep = A.c(), B.c(), _epilogue(bias, act)
    ldc = out.stride(0)
    _check(lib().mx_gemm_fused(ctypes.byref(ca), ctypes.byref(cb),
                               ctypes.byref(ep),
                               out.data_ptr() if out.numel() else None, dt,
                               ldc, _stream(stream)), "mx_gemm_fused")
    return out


def mx_gemm_fused_quantize(A: MXTensor, B: MXTensor, fmt: int,
                           bias: torch.Tensor | None = None,
                           act: int = ACT_NONE, out: MXTensor | None = None,
                           stream=None) -> MXTensor:
    """act(A * B + bias) quantized in the GEMM epilogue to an M x N MX
    tensor (blocks of 32 along N) of element format fmt."""
    _check_bias(bias, B.outer)
    _check_mx(A, "A")
    _check_mx(B, "B")
    if out is None:
        out = empty_mx(fmt, A.outer, B.outer, A.data.device)
    _check_mx(out, "out", fmt, A.outer, B.outer)
    ca, cb, cc, ep = A.c(), B.c(), out.c(), _epilogue(bias, act)
    _check(lib().mx_gemm_fused_quantize(ctypes.byref(ca), ctypes.byref(cb),
                                        ctypes.byref(ep), ctypes.byref(cc),
                                        _stream(stream)),
           "mx_gemm_fused_quantize")
    return out


def gemm_f16_fused(A: torch.Tensor, B: torch.Tensor,
                   bias: torch.Tensor | None = None, act: int = ACT_NONE,
                   out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """C (fp32) = act(A * B + bias) for row-major fp16 or bf16 tensors."""
    if A.dtype != B.dtype or A.dtype not in (torch.float16, torch.bfloat16):
        raise ValueError("A and B must both be fp16 or both bf16")
    M, K = A.shape
    K2, N = B.shape
    if K != K2:
        raise ValueError("inner dimensions differ")
    _check_bias(bias, N)
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=A.device)
    _check_out(out, M, N, torch.float32)
    dt = DT_F16 if A.dtype == torch.float16 else DT_BF16
    ep = _epilogue(bias, act)
    _check(lib().gemm_f16_fused(
        A.data_ptr() if A.numel() else None,
        B.data_ptr() if B.numel() else None, ctypes.byref(ep),
        out.data_ptr() if out.numel() else None, dt, M, N, K, A.stride(0),
        B.stride(0), out.stride(0), _stream(stream)), "gemm_f16_fused")
    return out


def gemm_dequant_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib().gemm_dequant_workspace_bytes(M, N, K))


def gemm_dequant(A: torch.Tensor, B: MXTensor, bias: torch.Tensor | None = None,
                 act: int = ACT_NONE, out_dtype=torch.float32,
                 out: torch.Tensor | None = None, stream=None,
                 workspace: torch.Tensor | None = None) -> torch.Tensor:
    """C = act(A * dequant(B)^T + bias) for a row-major fp16 / bf16 A
    (M x K) and an MX tensor B of any format (N x K, quantized from a K x N
    matrix): B is dequantized to A's type in shared or tensor memory, or in
    registers for a single bf16 row with 4- or 2-bit codes.  With a
    workspace (gemm_dequant_workspace_bytes) the K-split entry point runs."""
    if A.dtype not in (torch.float16, torch.bfloat16) or A.dim() != 2:
        raise ValueError("A must be a 2-D fp16 or bf16 tensor")
    if A.stride(1) != 1:
        raise ValueError("A must have a unit inner stride")
    M, K = A.shape
    if K != B.K:
        raise ValueError("inner dimensions differ")
    _check_bias(bias, B.outer)
    dt = _out_code(out_dtype, (torch.float32, torch.bfloat16))
    _check_mx(B, "B")
    if out is None:
        out = torch.empty((M, B.outer), dtype=out_dtype, device=A.device)
    _check_out(out, M, B.outer, out_dtype)
    cb, ep = B.c(), _epilogue(bias, act)
    args = (A.data_ptr() if A.numel() else None,
            DT_F16 if A.dtype == torch.float16 else DT_BF16, M, A.stride(0),
            ctypes.byref(cb), ctypes.byref(ep),
            out.data_ptr() if out.numel() else None, dt,
            out.stride(0))
    if workspace is None:
        _check(lib().gemm_dequant(*args, _stream(stream)), "gemm_dequant")
    else:
        _check(lib().gemm_dequant_splitk(
            *args, workspace.data_ptr() if workspace.numel() else None,
            _nbytes(workspace), _stream(stream)),
            "gemm_dequant_splitk")
    return out


def flash_attention(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor,
                    scale: float | None = None, out_dtype=torch.float32,
                    out: torch.Tensor | None = None, stream=None,
                    workspace: torch.Tensor | None = None) -> torch.Tensor:
    """O = softmax(Q K^T * scale) V per head.  Q is (..., Lq, d), K and V
    (..., Lk, d), contiguous fp16 or bf16 CUDA tensors with the same leading
    dimensions (flattened into heads); scale defaults to 1/sqrt(d).  With a
    device `workspace` (uint8, flash_attention_workspace_bytes() long) the
    key axis is split over SMs that would otherwise idle."""
    if Q.dtype not in (torch.float16, torch.bfloat16) or K.dtype != Q.dtype \
            or V.dtype != Q.dtype:
        raise ValueError("Q, K, V must share an fp16 or bf16 dtype")
    if not (Q.is_contiguous() and K.is_contiguous() and V.is_contiguous()):
        raise ValueError("Q, K, V must be contiguous")
    if K.shape != V.shape or Q.shape[:-2] != K.shape[:-2] or \
            Q.shape[-1] != K.shape[-1]:
        raise ValueError("shape mismatch")
    Lq, d = Q.shape[-2], Q.shape[-1]
    Lk = K.shape[-2]
    BH = Q.numel() // max(1, Lq * d)
    if scale is None:
        scale = 1.0 / float(d) ** 0.5
    odt = _out_code(out_dtype, (torch.float32, torch.bfloat16, torch.float16))
    if out is None:
        out = torch.empty(Q.shape, dtype=out_dtype, device=Q.device)
    if (out.dtype != out_dtype or not out.is_cuda or out.shape != Q.shape
            or not out.is_contiguous()):
        raise ValueError("out must be a contiguous CUDA tensor of Q's shape "
                         "and type out_dtype")
    ptr = lambda t: t.data_ptr() if t.numel() else None  # noqa
    dt = DT_F16 if Q.dtype == torch.float16 else DT_BF16
    if workspace is None:
        _check(lib().flash_attention(
            ptr(Q), ptr(K), ptr(V), ptr(out), dt, odt, BH, Lq, Lk, d,
            float(scale), _stream(stream)), "flash_attention")
    else:
        _check(lib().flash_attention_splitkv(
            ptr(Q), ptr(K), ptr(V), ptr(out), dt, odt, BH, Lq, Lk, d,
            float(scale), ptr(workspace), _nbytes(workspace), _stream(stream)),
            "flash_attention_splitkv")
    return out


def flash_attention_workspace_bytes(BH: int, Lq: int, Lk: int, d: int) -> int:
    """Bytes of workspace flash_attention splits into (0: no split)."""
    return int(lib().flash_attention_workspace_bytes(BH, Lq, Lk, d))


@dataclass
class KVCache:
    """An 8-bit paged key/value cache: code planes (uint8, pages x heads x page
    x d), one UE8M0 scale byte for each page and head (uint8, pages x heads),
    and the element format (E4M3, E5M2 or INT8)."""
    k: torch.Tensor
    v: torch.Tensor
    k_scales: torch.Tensor
    v_scales: torch.Tensor
    fmt: int

    def __post_init__(self):
        shape = self.k.shape
        if len(shape) != 4 or self.v.shape != shape:
            raise ValueError("k and v must be pages x heads x page x d")
        if self.k_scales.shape != shape[:2] or self.v_scales.shape != shape[:2]:
            raise ValueError("scales must be pages x heads")
        for t in (self.k, self.v, self.k_scales, self.v_scales):
            if t.dtype != torch.uint8 or not t.is_contiguous():
                raise ValueError("a cache's planes are contiguous uint8 tensors")
        # one GPU's memory: the calls ask, a cache on the host may be kept
        self._gpu = self.k.is_cuda and all(
            t.device == self.k.device for t in (self.v, self.k_scales, self.v_scales))
        pages, heads, page, d = shape
        self._c = CKVCache(self.k.data_ptr(), self.v.data_ptr(),
                           self.k_scales.data_ptr(), self.v_scales.data_ptr(),
                           self.fmt, page, pages, heads, d)
        self._of = self._planes()

    def __getstate__(self):                      # copies have addresses of their own
        return {f: getattr(self, f) for f in self.__dataclass_fields__}

    def __setstate__(self, state):
        self.__dict__.update(state)
        self.__post_init__()

    def _planes(self):
        """All that the C struct follows from."""
        k, v, ks, vs = self.k, self.v, self.k_scales, self.v_scales
        return (self.fmt, k.data_ptr(), v.data_ptr(), ks.data_ptr(),
                vs.data_ptr(), k.shape, v.shape, ks.shape, vs.shape,
                k.is_contiguous(), v.is_contiguous(), ks.is_contiguous(),
                vs.is_contiguous())

    def c(self) -> CKVCache:
        """The planes as they are now, checked again if any of them changed."""
        if self._of != self._planes():
            self.__post_init__()
        return self._c

    def on_gpu(self) -> CKVCache:
        """c(), for a call that follows its addresses on the GPU."""
        c = self.c()
        if not self._gpu:
            raise ValueError("a cache's planes must be CUDA tensors of one GPU")
        return c


def empty_kv_cache(fmt: int, pages: int, heads: int, page: int, d: int,
                   device="cuda") -> KVCache:
    """A cache of uninitialised pages: a page means nothing until its first
    token is appended."""
    def u8(*shape):
        return torch.empty(shape, dtype=torch.uint8, device=device)
    return KVCache(u8(pages, heads, page, d), u8(pages, heads, page, d),
                   u8(pages, heads), u8(pages, heads), fmt)


@dataclass
class KVPlan:
    """What mx_kv_extend gives: the requests' new lengths, the offsets of
    their new tokens, the tokens' slots, and [free pages, requests refused]."""
    lens: torch.Tensor
    cu: torch.Tensor
    slots: torch.Tensor
    counts: torch.Tensor


@dataclass
class KVCut:
    """What mx_kv_truncate gives: the new lengths, and [free pages, pages the
    stack had no room for]."""
    lens: torch.Tensor
    counts: torch.Tensor


# The cache's calls take a few microseconds on the GPU in a decoding step, less
# than careful Python around them: shapes and strides are read once, and
# dtypes looked up in tables.
_i32 = torch.int32
_KV_DTYPES = {torch.float16: DT_F16, torch.bfloat16: DT_BF16}
_KV_OUT_DTYPES = {torch.float32: DT_F32, torch.bfloat16: DT_BF16,
                  torch.float16: DT_F16}


# An uninitialised tensor on the current GPU: (shape, strides, dtype).  The
# allocator's entry without the operator dispatch around it, whose code a
# kernel launch between two calls pushes out of the host's caches: 3.6 us
# instead of 7 in a decoding step.  It is not public: None where torch lacks it.
try:
    _direct_empty = torch._C._dynamo.guards._empty_strided_cuda
except AttributeError:
    _direct_empty = None


def _allocator(like: torch.Tensor):
    """What makes a call's outputs, on the operands' GPU: the direct entry where
    that is the current one, torch.empty_strided on another, without that entry
    and where torch is to fill what nothing writes."""
    if _direct_empty is not None and \
            like.get_device() == torch.cuda.current_device() and \
            not torch.are_deterministic_algorithms_enabled():
        return _direct_empty
    device = like.device
    return lambda shape, strides, dtype: torch.empty_strided(
        shape, strides, dtype=dtype, device=device)


def _int32(t: torch.Tensor, name: str, n: int = 0) -> int:
    """Checks a vector of int32 values; its address."""
    if t.dtype is not _i32 or not t.is_cuda or t.dim() != 1 or \
            not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 1-D int32 CUDA tensor")
    if t.numel() < n:
        raise ValueError(f"{name} must hold {n} values")
    return t.data_ptr()


def _table(table: torch.Tensor, requests: int) -> tuple[int, int, int]:
    """Checks a block table; its address, row stride and width."""
    shape, stride = table.shape, table.stride()
    if table.dtype is not _i32 or not table.is_cuda or len(shape) != 2 or \
            shape[0] < requests:
        raise ValueError("table must be a 2-D int32 CUDA tensor with a row for "
                         "each request")
    width = shape[1]
    if width > 1 and stride[1] != 1:
        raise ValueError("table must have a unit inner stride")
    # the stride of a dimension of size 1 means nothing
    return (table.data_ptr(),
            stride[0] if shape[0] > 1 else max(stride[0], width), width)


def mx_kv_extend(lens: torch.Tensor, new_tokens: torch.Tensor,
                 table: torch.Tensor, stack: torch.Tensor, count: torch.Tensor,
                 page: int, max_tokens: int, out: KVPlan | None = None,
                 stream=None) -> KVPlan:
    """Room for new tokens: pages from the stack of free ones into the
    requests' rows of the block table (in place), and every new token's slot.
    lens, new_tokens: int32, one per request; table: int32, requests x width;
    stack, count: the free pages' ids and, in count[0], their number;
    max_tokens: the most new tokens there may be (the length of slots).  A
    request that finds no room, and every one behind it, is refused whole."""
    B = lens.shape[0]
    p_lens = _int32(lens, "lens")
    p_new = _int32(new_tokens, "new_tokens", B)
    p_stack = _int32(stack, "stack")
    p_count = _int32(count, "count", 1)
    p_table, stride, width = _table(table, B)
    if out is None:
        one, empty = (1,), _allocator(lens)
        out = KVPlan(empty((B,), one, _i32), empty((B + 1,), one, _i32),
                     empty((max_tokens,), one, torch.int64),
                     empty((2,), one, _i32))
    else:
        _int32(out.lens, "out.lens", B)
        _int32(out.cu, "out.cu", B + 1)
        _int32(out.counts, "out.counts", 2)
        if out.slots.dtype != torch.int64 or not out.slots.is_cuda or \
                not out.slots.is_contiguous() or out.slots.numel() < max_tokens:
            raise ValueError("out.slots must hold max_tokens int64 values")
    _check(lib().mx_kv_extend(
        p_lens, p_new, B, p_table, stride, width, p_stack, stack.numel(),
        p_count, page, out.lens.data_ptr(), out.cu.data_ptr(),
        out.slots.data_ptr(), max_tokens, out.counts.data_ptr(),
        _stream(stream)), "mx_kv_extend")
    return out


def mx_kv_truncate(lens: torch.Tensor, keep: torch.Tensor, table: torch.Tensor,
                   stack: torch.Tensor, count: torch.Tensor, page: int,
                   out: KVCut | None = None, stream=None) -> KVCut:
    """Drop tokens from the ends of requests: request b keeps keep[b] of its
    tokens (0: it is finished).  Pages that become free go back on the stack
    (in place) and their table entries become -1; an mx_kv_extend by as many
    tokens hands out the same pages again."""
    B = lens.shape[0]
    p_lens = _int32(lens, "lens")
    p_keep = _int32(keep, "keep", B)
    p_stack = _int32(stack, "stack")
    p_count = _int32(count, "count", 1)
    p_table, stride, width = _table(table, B)
    if out is None:
        empty = _allocator(lens)
        out = KVCut(empty((B,), (1,), _i32), empty((2,), (1,), _i32))
    else:
        _int32(out.lens, "out.lens", B)
        _int32(out.counts, "out.counts", 2)
    _check(lib().mx_kv_truncate(
        p_lens, p_keep, B, p_table, stride, width, p_stack, stack.numel(),
        p_count, page, out.lens.data_ptr(), out.counts.data_ptr(),
        _stream(stream)), "mx_kv_truncate")
    return out


def _kv_tensor(t: torch.Tensor, name: str):
    """Checks a tokens x heads x d tensor; its type's code, shape, token stride
    and head stride (0 for a dimension of size 1, whose stride means
    nothing)."""
    dt, shape, stride = _KV_DTYPES.get(t.dtype), t.shape, t.stride()
    if dt is None or not t.is_cuda or len(shape) != 3:
        raise ValueError(f"{name} must be a tokens x heads x d fp16 or bf16 "
                         "CUDA tensor")
    if stride[2] != 1 and shape[2] > 1:
        raise ValueError(f"{name} must have a unit inner stride")
    return (dt, shape, stride[0] if shape[0] > 1 else 0,
            stride[1] if shape[1] > 1 else 0)


def mx_kv_append(cache: KVCache, K: torch.Tensor, V: torch.Tensor,
                 slots: torch.Tensor, stream=None) -> KVCache:
    """Quantize new keys and values (tokens x heads x d, fp16 or bf16) into the
    cache, in place, at their slots (int64, one per token; negative: none).
    One power-of-two scale covers a page and head: where new tokens need a
    larger one than the page has, the codes already there are rounded again."""
    c = cache.on_gpu()
    dt, shape, kt, kh = _kv_tensor(K, "K")
    vdt, vshape, vt, vh = _kv_tensor(V, "V")
    if vdt != dt or vshape != shape:
        raise ValueError("K and V must have one shape and type")
    T, heads, d = shape
    if heads != c.heads or d != c.d:
        raise ValueError("K and V must have the cache's heads and d")
    if slots.dtype != torch.int64 or not slots.is_cuda or slots.dim() != 1 or \
            not slots.is_contiguous() or slots.numel() < T:
        raise ValueError("slots must be a contiguous int64 CUDA tensor, one "
                         "for each token")
    _check(lib().mx_kv_append(ctypes.byref(c), K.data_ptr(), V.data_ptr(), dt,
                              T, kt, kh, vt, vh, slots.data_ptr(),
                              _stream(stream)), "mx_kv_append")
    return cache


def kv_attention_workspace_bytes(q_heads: int, heads: int, d: int,
                                 max_q: int) -> int:
    """Bytes of workspace with which mx_kv_attention spreads a request's keys
    over many SMs; the same for all lengths and numbers of requests."""
    return int(lib().mx_kv_attention_workspace_bytes(q_heads, heads, d, max_q))


def mx_kv_attention(Q: torch.Tensor, cache: KVCache, table: torch.Tensor,
                    lens: torch.Tensor, cu: torch.Tensor, max_q: int,
                    causal: bool = True, window: int = 0,
                    scale: float | None = None, out_dtype=None,
                    out: torch.Tensor | None = None, stream=None,
                    workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of the requests' last tokens over the cache.  Q: tokens x
    heads x d, fp16 or bf16, the rows of request b being cu[b] .. cu[b+1];
    lens: the requests' lengths, those rows included; max_q: the most rows
    any request has (or more).  causal: a row sees no key behind its own
    position; window > 0: and only the last `window` of those.  scale
    defaults to 1/sqrt(d), out_dtype to Q's.  With a device `workspace`
    (uint8, kv_attention_workspace_bytes() long) a request's keys are spread
    over many SMs.  Rows that belong to no request are not written."""
    if workspace is not None and not (workspace.is_cuda and
                                      workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor")
    c = cache.on_gpu()
    dt, shape, qt, qh = _kv_tensor(Q, "Q")
    T, Hq, d = shape
    if d != c.d or Hq % c.heads:
        raise ValueError("Q must have the cache's d and a multiple of its heads")
    B = lens.shape[0]
    p_lens = _int32(lens, "lens")
    p_cu = _int32(cu, "cu", B + 1)
    p_table, stride, width = _table(table, B)
    if out is None:
        ot, oh = Hq * d, d
        out = _allocator(Q)((T, Hq, d), (ot, oh, 1), out_dtype or Q.dtype)
    elif (out.shape != shape or not out.is_cuda or out.stride(2) != 1
          or (out_dtype is not None and out.dtype != out_dtype)):
        raise ValueError("out must be a CUDA tensor of Q's shape and of type "
                         "out_dtype, with a unit inner stride")
    else:
        ot = out.stride(0) if T > 1 else 0
        oh = out.stride(1) if Hq > 1 else 0
    odt = _KV_OUT_DTYPES.get(out.dtype)
    if odt is None:
        raise ValueError("out_dtype must be float32, bfloat16 or float16, not "
                         f"{out.dtype}")
    _check(lib().mx_kv_attention(
        Q.data_ptr(), dt, T, Hq, qt, qh, ctypes.byref(c), p_table, stride,
        width, p_lens, p_cu, B, max_q, out.data_ptr(), odt, ot, oh,
        1 if causal else 0, window, d ** -0.5 if scale is None else scale,
        None if workspace is None else workspace.data_ptr(),
        _nbytes(workspace), _stream(stream)), "mx_kv_attention")
    return out


def mx_last_error(stream=None) -> int:
    """Synchronize the stream and return (and clear) the library's device
    status (0 = MX_OK, 6 = MX_ERR_TIMEOUT)."""
    return int(lib().mx_last_error(_stream(stream)))


def mx_selftest_wait_timeout(limit_cycles: int, stream=None) -> int:
    return int(lib().mx_selftest_wait_timeout(limit_cycles, _stream(stream)))


def scales_to_rowmajor(tiled, outer: int, K: int):
    """Host helper: tiled scale plane (numpy uint8) -> outer x K/32 array."""
    import numpy as np
    t = np.ascontiguousarray(tiled, dtype=np.uint8)
    out = np.empty((outer, K // 32), dtype=np.uint8)
    _check(lib().mx_scales_to_rowmajor(t.ctypes.data, out.ctypes.data, outer,
                                       K), "mx_scales_to_rowmajor")
    return out


def set_tile_width(tbn: int) -> None:
    """Fix the GEMMs' output-tile width (128 or 256) for later calls, or let
    the library pick it per shape (0, the default)."""
    _check(lib().mx_set_tile_width(int(tbn)), "mx_set_tile_width")
