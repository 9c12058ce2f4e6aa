"""Python binding of libqlora: NF4 + double-quant frozen linear layer with LoRA on B200.

A thin ctypes layer over the C ABI in ``include/qlora.h``.  It only marshals
arguments -- device pointers of torch tensors, sizes, the current CUDA stream --
and allocates the output tensors and work buffers with torch.  Every step of the
computation runs in the library's sm_100a kernels; there is no CPU fallback:
if ``libqlora.so`` is missing or fails to load, importing this module raises.

Entry points (same names as the C ABI):
    qlora_quantize_nf4_dq(W)                          -> NF4Tensor
    qlora_dequantize(qt)                              -> bf16 [rows, cols]
    qlora_linear_fwd(qt, X, A, B, s, save_xa=True)    -> (Y bf16, XA fp32 or None)
    qlora_linear_fwd_multi(qt, X, A_stack, B_stack, adapter_idx, s) -> (Y, XA): one adapter per token
    qlora_linear_bwd(qt, X, dY, A, B, s, XA=None, need_dx=True) -> (dX bf16 or None, dA fp32, dB fp32)
    qlora_get_codebook()                              -> 16 float levels
Microscaled 4-bit formats (MXFP4, NVFP4):
    qlora_mx_quantize(W, fmt, transpose, per_row)     -> MXTensor
    qlora_mx_dequantize(q)                            -> bf16 [rows, cols]
    qlora_mx_linear_fwd(q, X, A, B, s)                -> (Y bf16, XA fp32 or None)
    qlora_mx_linear_bwd(qT, dY, X, A, B, s, XA)       -> (dX bf16 or None, dA fp32, dB fp32)
    qlora_mx_moe_fwd(W13, W2, router, X, top_k)       -> (Y bf16, ids int32, probs fp32): experts for a few tokens
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqlora.so")

BLOCKSIZE = 64
BLOCKSIZE2 = 256

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libqlora.so not built at {LIB_PATH}; run "
                      "`python bit_nf4_quantized_encode_b200/build.py` (nvcc, sm_100a)")
_lib = ctypes.CDLL(LIB_PATH)


class _Nf4TensorC(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("absmax_q", ctypes.c_void_p),
                ("absmax_c2", ctypes.c_void_p), ("absmax_mean", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("blocksize", ctypes.c_int32), ("blocksize2", ctypes.c_int32),
                ("absmax", ctypes.c_void_p), ("quant_type", ctypes.c_int32), ("reserved", ctypes.c_int32)]


# The 4-bit data types (qlora_quant_type): NF4 and the two it is compared with.
QUANT_TYPES = {"nf4": 0, "fp4": 1, "int4": 2}


_vp, _i64, _i32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
_szp = ctypes.POINTER(ctypes.c_size_t)
_T = ctypes.POINTER(_Nf4TensorC)

_lib.qlora_status_string.argtypes = [ctypes.c_int]
_lib.qlora_status_string.restype = ctypes.c_char_p
_lib.qlora_get_codebook.argtypes = [ctypes.POINTER(ctypes.c_float)]
_lib.qlora_get_codebook.restype = None
_lib.qlora_get_levels.argtypes = [_i32, ctypes.POINTER(ctypes.c_float)]
_lib.qlora_get_levels.restype = ctypes.c_int
_lib.qlora_nf4_sizes.argtypes = [_i64, _i64, _i32, _i32, _szp, _szp, _szp, _szp]
_lib.qlora_nf4_sizes.restype = ctypes.c_int
_lib.qlora_quantize_nf4_dq.argtypes = [_vp, _T, _vp, _sz, _vp]
_lib.qlora_quantize_nf4_dq.restype = ctypes.c_int
_lib.qlora_dequantize.argtypes = [_T, _vp, _vp]
_lib.qlora_dequantize.restype = ctypes.c_int
_lib.qlora_linear_workspace_size.argtypes = [_i64, _i64, _i64, _i32, _szp, _szp]
_lib.qlora_linear_workspace_size.restype = ctypes.c_int
_lib.qlora_linear_fwd.argtypes = [_T, _vp, _i64, _vp, _vp, _i32, ctypes.c_float, _vp, _vp, _vp,
                                  _sz, _vp]
_lib.qlora_linear_fwd.restype = ctypes.c_int
_lib.qlora_linear_fwd_multi.argtypes = [_T, _vp, _i64, _vp, _vp, _i32, _vp, _i32, ctypes.c_float, _vp, _vp,
                                        _vp, _sz, _vp]
_lib.qlora_linear_fwd_multi.restype = ctypes.c_int
_lib.qlora_linear_bwd.argtypes = [_T, _vp, _vp, _i64, _vp, _vp, _i32, ctypes.c_float, _vp, _vp,
                                  _vp, _vp, _vp, _sz, _vp]
_lib.qlora_linear_bwd.restype = ctypes.c_int
_lib.qlora_read_device_errors.argtypes = [ctypes.POINTER(ctypes.c_uint32), ctypes.c_int]
_lib.qlora_read_device_errors.restype = ctypes.c_int
_lib.qlora_quantize_nf4_dq_noalloc.argtypes = [_vp, _T, _vp]
_lib.qlora_quantize_nf4_dq_noalloc.restype = ctypes.c_int
_lib.qlora_kernel_launches.argtypes = []
_lib.qlora_kernel_launches.restype = ctypes.c_uint64
_lib.qlora_time_next_gemm.argtypes = [_vp, _vp]
_lib.qlora_time_next_gemm.restype = ctypes.c_int
_lib.qlora_selftest_bounded_wait.argtypes = [_i64, _vp, _vp]
_lib.qlora_selftest_bounded_wait.restype = ctypes.c_int

class _MxTensorC(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("global_scale", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("format", ctypes.c_int32), ("scale_per_row", ctypes.c_int32)]


_MX = ctypes.POINTER(_MxTensorC)
_lib.qlora_mx_sizes.argtypes = [_i64, _i64, _i32, _i32, _szp, _szp, _szp, _szp]
_lib.qlora_mx_sizes.restype = ctypes.c_int
_lib.qlora_mx_quantize.argtypes = [_vp, _i32, _MX, _vp, _sz, _vp]
_lib.qlora_mx_quantize.restype = ctypes.c_int
_lib.qlora_mx_dequantize.argtypes = [_MX, _vp, _vp]
_lib.qlora_mx_dequantize.restype = ctypes.c_int
_lib.qlora_mx_linear_workspace_size.argtypes = [_i64, _i64, _i32, _i64, _i32, _szp, _szp]
_lib.qlora_mx_linear_workspace_size.restype = ctypes.c_int
_lib.qlora_mx_linear_fwd.argtypes = [_MX, _vp, _i64, _vp, _vp, _i32, ctypes.c_float, _vp, _vp, _vp, _sz, _vp]
_lib.qlora_mx_linear_fwd.restype = ctypes.c_int
_lib.qlora_mx_linear_bwd.argtypes = [_MX, _vp, _vp, _i64, _vp, _vp, _i32, ctypes.c_float, _vp, _vp, _vp, _vp, _vp,
                                     _sz, _vp]
_lib.qlora_mx_linear_bwd.restype = ctypes.c_int
_lib.qlora_mx_moe_workspace_size.argtypes = [_i32, _i64, _i64, _i64, _i32, _szp]
_lib.qlora_mx_moe_workspace_size.restype = ctypes.c_int
_lib.qlora_mx_moe_fwd.argtypes = [_MX, _MX, _vp, _i32, _vp, _i64, _i32, _vp, _vp, _vp, _vp, _sz, _vp]
_lib.qlora_mx_moe_fwd.restype = ctypes.c_int
_lib.qlora_selftest_mx_form.argtypes = [_i64, _i64, _i32, _i64, _i32, _i32, _i32, ctypes.POINTER(_i32), ctypes.POINTER(_i32)]
_lib.qlora_selftest_mx_form.restype = ctypes.c_int

EXPORTED = ["qlora_status_string", "qlora_get_codebook", "qlora_get_levels", "qlora_nf4_sizes", "qlora_quantize_nf4_dq",
            "qlora_dequantize", "qlora_linear_workspace_size", "qlora_linear_fwd", "qlora_linear_fwd_multi",
            "qlora_linear_bwd", "qlora_read_device_errors", "qlora_kernel_launches",
            "qlora_time_next_gemm", "qlora_quantize_nf4_dq_noalloc", "qlora_selftest_bounded_wait",
            "qlora_mx_sizes", "qlora_mx_quantize", "qlora_mx_dequantize",
            "qlora_mx_linear_workspace_size", "qlora_mx_linear_fwd", "qlora_mx_linear_bwd",
            "qlora_mx_moe_workspace_size", "qlora_mx_moe_fwd", "qlora_selftest_mx_form"]

# Largest weight the allocation-free quantize variant accepts.
NOALLOC_MAX_ELEMENTS = 134217728


class QloraError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib.qlora_status_string(status).decode()
        super().__init__(f"{where}: {msg} (status {status})")


def _check(status: int, where: str):
    if status != 0:
        raise QloraError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need_bf16_cuda(name: str, t: torch.Tensor):
    if not (t.is_cuda and t.dtype == torch.bfloat16 and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous bf16 CUDA tensor")


@dataclass
class NF4Tensor:
    """A quantized weight: packed 4-bit codes and its block constants, stored
    either double-quantized (E4M3 codes, c2 per group, mean) or as fp32 absmax
    per block (`absmax`, no double quantization)."""
    codes: torch.Tensor                     # uint8 [ceil(rows*cols/2)]
    absmax_q: torch.Tensor | None           # uint8 [ceil(rows*cols/64)] (double quantization)
    absmax_c2: torch.Tensor | None          # float32 [ceil(nblocks/256)] (double quantization)
    absmax_mean: torch.Tensor | None        # float32 [1] (double quantization)
    rows: int
    cols: int
    absmax: torch.Tensor | None = None      # float32 [nblocks] (no double quantization)
    quant_type: str = "nf4"                 # "nf4", "fp4" or "int4"

    @property
    def double_quant(self) -> bool:
        return self.absmax is None

    def c_struct(self) -> _Nf4TensorC:
        p = lambda t: 0 if t is None else t.data_ptr()
        return _Nf4TensorC(self.codes.data_ptr(), p(self.absmax_q), p(self.absmax_c2), p(self.absmax_mean),
                           self.rows, self.cols, BLOCKSIZE, BLOCKSIZE2 if self.double_quant else 0,
                           p(self.absmax), QUANT_TYPES[self.quant_type], 0)

    def buffers(self) -> dict:
        return {n: t for n, t in (("codes", self.codes), ("absmax_q", self.absmax_q),
                                  ("absmax_c2", self.absmax_c2), ("absmax_mean", self.absmax_mean),
                                  ("absmax", self.absmax)) if t is not None}

    @property
    def device(self):
        return self.codes.device

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in self.buffers().values())


def qlora_status_string(status: int) -> str:
    return _lib.qlora_status_string(int(status)).decode()


def qlora_get_codebook() -> list:
    out = (ctypes.c_float * 16)()
    _lib.qlora_get_codebook(out)
    return list(out)


def qlora_get_levels(quant_type: str = "nf4") -> list:
    """The 16 levels of a 4-bit type ("nf4", "fp4" or "int4")."""
    out = (ctypes.c_float * 16)()
    _check(_lib.qlora_get_levels(QUANT_TYPES[quant_type], out), "qlora_get_levels")
    return list(out)


def qlora_nf4_sizes(rows: int, cols: int, double_quant: bool = True) -> dict:
    """Buffer sizes in bytes; without double quantization 'absmax_q' is the
    size of the fp32 absmax array and 'absmax_c2' is 0."""
    v = [ctypes.c_size_t() for _ in range(4)]
    _check(_lib.qlora_nf4_sizes(rows, cols, BLOCKSIZE, BLOCKSIZE2 if double_quant else 0,
                                *[ctypes.byref(x) for x in v]), "qlora_nf4_sizes")
    return dict(codes=v[0].value, absmax_q=v[1].value, absmax_c2=v[2].value, workspace=v[3].value)


def empty_nf4(rows: int, cols: int, device, quant_type: str = "nf4", double_quant: bool = True) -> NF4Tensor:
    if quant_type not in QUANT_TYPES:
        raise ValueError(f"quant_type must be one of {sorted(QUANT_TYPES)}")
    sz = qlora_nf4_sizes(rows, cols, double_quant)
    # round each buffer up to 16 bytes so every pointer the library sees is aligned
    def buf(n, dtype, esize):
        return torch.empty(max(1, (n + 15) // 16 * 16 // esize), dtype=dtype, device=device)
    codes = buf(sz["codes"], torch.uint8, 1)
    if not double_quant:
        return NF4Tensor(codes=codes, absmax_q=None, absmax_c2=None, absmax_mean=None, rows=rows, cols=cols,
                         absmax=buf(sz["absmax_q"], torch.float32, 4), quant_type=quant_type)
    return NF4Tensor(codes=codes, absmax_q=buf(sz["absmax_q"], torch.uint8, 1),
                     absmax_c2=buf(sz["absmax_c2"], torch.float32, 4),
                     absmax_mean=torch.empty(4, dtype=torch.float32, device=device),
                     rows=rows, cols=cols, quant_type=quant_type)


def _check_out_matches(W: torch.Tensor, out: NF4Tensor):
    """The C entry points take the shape from `out` alone and read that many
    weights from W: refuse a destination that describes another tensor."""
    if out.rows * out.cols != W.numel():
        raise ValueError(f"out describes {out.rows}x{out.cols} weights, W has {W.numel()}")
    for name, t in out.buffers().items():
        if t.device != W.device:
            raise ValueError(f"out.{name} is on {t.device}, W on {W.device}")


def qlora_quantize_nf4_dq(W: torch.Tensor, out: NF4Tensor | None = None,
                          workspace: torch.Tensor | None = None, quant_type: str = "nf4",
                          double_quant: bool = True) -> NF4Tensor:
    """Blockwise 4-bit encode (NF4 by default) + double quantization of a bf16
    [rows, cols] weight; `out`, when given, fixes the type and the form."""
    _need_bf16_cuda("W", W)
    rows, cols = (W.shape[0], W.shape[1]) if W.dim() == 2 else (1, W.numel())
    if out is None:
        out = empty_nf4(rows, cols, W.device, quant_type, double_quant)
    _check_out_matches(W, out)
    need = qlora_nf4_sizes(out.rows, out.cols, out.double_quant)["workspace"]
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=W.device)
    c = out.c_struct()
    _check(_lib.qlora_quantize_nf4_dq(_ptr(W), ctypes.byref(c), _ptr(workspace),
                                      workspace.numel(), _stream(W.device)), "qlora_quantize_nf4_dq")
    return out


def qlora_quantize_nf4_dq_noalloc(W: torch.Tensor, out: NF4Tensor) -> NF4Tensor:
    """Same result as qlora_quantize_nf4_dq, with the library's built-in scratch
    instead of a work buffer (for callers that cannot allocate; see qlora.h)."""
    _need_bf16_cuda("W", W)
    _check_out_matches(W, out)
    c = out.c_struct()
    _check(_lib.qlora_quantize_nf4_dq_noalloc(_ptr(W), ctypes.byref(c), _stream(W.device)),
           "qlora_quantize_nf4_dq_noalloc")
    return out


def qlora_dequantize(qt: NF4Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """Two-level dequantization to a bf16 [rows, cols] tensor."""
    if out is None:
        out = torch.empty(qt.rows, qt.cols, dtype=torch.bfloat16, device=qt.device)
    c = qt.c_struct()
    _check(_lib.qlora_dequantize(ctypes.byref(c), _ptr(out), _stream(qt.device)), "qlora_dequantize")
    return out


def qlora_linear_workspace_size(rows: int, cols: int, m: int, r: int) -> tuple:
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    _check(_lib.qlora_linear_workspace_size(rows, cols, m, r, ctypes.byref(f), ctypes.byref(b)),
           "qlora_linear_workspace_size")
    return f.value, b.value


def qlora_linear_fwd(qt: NF4Tensor, X: torch.Tensor, A: torch.Tensor, B: torch.Tensor, s: float,
                     save_xa: bool = True, Y: torch.Tensor | None = None,
                     XA: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """Y = X deq(W)^T + s (X A^T) B^T.  Returns (Y bf16, XA) with XA = X A^T in fp32 (or None)."""
    for n, t in (("X", X), ("A", A), ("B", B)):
        _need_bf16_cuda(n, t)
    m, r = X.shape[0], A.shape[0]
    if Y is None:
        Y = torch.empty(m, qt.rows, dtype=torch.bfloat16, device=X.device)
    if save_xa and XA is None:
        XA = torch.empty(m, r, dtype=torch.float32, device=X.device)
    if workspace is None:
        workspace = torch.empty(qlora_linear_workspace_size(qt.rows, qt.cols, m, r)[0],
                                dtype=torch.uint8, device=X.device)
    c = qt.c_struct()
    _check(_lib.qlora_linear_fwd(ctypes.byref(c), _ptr(X), m, _ptr(A), _ptr(B), r, float(s), _ptr(Y),
                                 _ptr(XA if save_xa else None), _ptr(workspace), workspace.numel(),
                                 _stream(X.device)), "qlora_linear_fwd")
    return Y, (XA if save_xa else None)


def qlora_linear_fwd_multi(qt: NF4Tensor, X: torch.Tensor, A_stack: torch.Tensor, B_stack: torch.Tensor,
                           adapter_idx: torch.Tensor, s: float, save_xa: bool = True,
                           Y: torch.Tensor | None = None, XA: torch.Tensor | None = None,
                           workspace: torch.Tensor | None = None):
    """Decode-shaped forward (M <= 16) with one adapter per token:
    Y[t] = X[t] deq(W)^T + s (X[t] A_a^T) B_a^T with a = adapter_idx[t]
    (int32 on the device; negative = no adapter).  A_stack [n, r, cols] and
    B_stack [n, rows, r] bf16.  Returns (Y bf16, XA fp32 or None)."""
    for n, t in (("X", X), ("A_stack", A_stack), ("B_stack", B_stack)):
        _need_bf16_cuda(n, t)
    if not (adapter_idx.is_cuda and adapter_idx.dtype == torch.int32 and adapter_idx.is_contiguous()
            and adapter_idx.numel() == X.shape[0]):
        raise ValueError("adapter_idx must be a contiguous int32 CUDA tensor with one entry per token")
    if A_stack.dim() != 3 or B_stack.dim() != 3 or A_stack.shape[0] != B_stack.shape[0]:
        raise ValueError("A_stack [n, r, cols] and B_stack [n, rows, r] must hold the same adapters")
    m, n_ad, r = X.shape[0], A_stack.shape[0], A_stack.shape[1]
    if Y is None:
        Y = torch.empty(m, qt.rows, dtype=torch.bfloat16, device=X.device)
    if save_xa and XA is None:
        XA = torch.empty(m, r, dtype=torch.float32, device=X.device)
    if workspace is None:
        workspace = torch.empty(qlora_linear_workspace_size(qt.rows, qt.cols, m, r)[0],
                                dtype=torch.uint8, device=X.device)
    c = qt.c_struct()
    _check(_lib.qlora_linear_fwd_multi(ctypes.byref(c), _ptr(X), m, _ptr(A_stack), _ptr(B_stack), n_ad,
                                       _ptr(adapter_idx), r, float(s), _ptr(Y), _ptr(XA if save_xa else None),
                                       _ptr(workspace), workspace.numel(), _stream(X.device)),
           "qlora_linear_fwd_multi")
    return Y, (XA if save_xa else None)


def qlora_linear_bwd(qt: NF4Tensor, X: torch.Tensor, dY: torch.Tensor, A: torch.Tensor,
                     B: torch.Tensor, s: float, XA: torch.Tensor | None = None, need_dx: bool = True,
                     dX: torch.Tensor | None = None, dA: torch.Tensor | None = None,
                     dB: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """Returns (dX bf16 or None, dA fp32, dB fp32) of the frozen-NF4 LoRA linear layer."""
    for n, t in (("X", X), ("dY", dY), ("A", A), ("B", B)):
        _need_bf16_cuda(n, t)
    m, r = X.shape[0], A.shape[0]
    dev = X.device
    if need_dx and dX is None:
        dX = torch.empty(m, qt.cols, dtype=torch.bfloat16, device=dev)
    if dA is None:
        dA = torch.empty(r, qt.cols, dtype=torch.float32, device=dev)
    if dB is None:
        dB = torch.empty(qt.rows, r, dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty(qlora_linear_workspace_size(qt.rows, qt.cols, m, r)[1],
                                dtype=torch.uint8, device=dev)
    c = qt.c_struct()
    _check(_lib.qlora_linear_bwd(ctypes.byref(c), _ptr(X), _ptr(dY), m, _ptr(A), _ptr(B), r,
                                 float(s), _ptr(XA), _ptr(dX if need_dx else None), _ptr(dA),
                                 _ptr(dB), _ptr(workspace), workspace.numel(), _stream(dev)),
           "qlora_linear_bwd")
    return (dX if need_dx else None), dA, dB


def qlora_read_device_errors(clear: bool = True) -> int:
    """Error flags set by kernels whose internal waits timed out (0 = none)."""
    v = ctypes.c_uint32()
    _check(_lib.qlora_read_device_errors(ctypes.byref(v), 1 if clear else 0),
           "qlora_read_device_errors")
    return v.value


def qlora_selftest_bounded_wait(limit_cycles: int, outcome: torch.Tensor | None = None) -> None:
    """Launch the failure-path self-test: one CTA whose bounded mbarrier wait
    must give up after `limit_cycles` SM cycles (see qlora.h)."""
    _check(_lib.qlora_selftest_bounded_wait(int(limit_cycles), _ptr(outcome),
                                            _stream(outcome.device if outcome is not None else None)),
           "qlora_selftest_bounded_wait")


def qlora_kernel_launches() -> int:
    """Kernels launched by the library in this process so far."""
    return int(_lib.qlora_kernel_launches())


def qlora_time_next_gemm(start: torch.cuda.Event, stop: torch.cuda.Event) -> None:
    """Bracket the calling thread's next fused dequant-GEMM launch with two CUDA events."""
    _check(_lib.qlora_time_next_gemm(ctypes.c_void_p(start.cuda_event), ctypes.c_void_p(stop.cuda_event)),
           "qlora_time_next_gemm")


# ---------------------------------------------------------------- microscaled 4-bit formats
# The formats (qlora_mx_format) and the elements of one of their blocks.
MX_FORMATS = {"mxfp4": 0, "nvfp4": 1}
MX_BLOCK = {"mxfp4": 32, "nvfp4": 16}


@functools.lru_cache(maxsize=4096)
def _mx_bytes(rows: int, cols: int, fmt: str) -> tuple:
    """(codes, scales) bytes of a microscaled matrix, as qlora_mx_sizes."""
    return rows * ((cols + 31) // 32 * 16), (rows + 127) // 128 * (-(-cols // (4 * MX_BLOCK[fmt]))) * 512


@dataclass
class MXTensor:
    """A microscaled 4-bit matrix: packed e2m1 codes, one scale byte per block
    of 32 (MXFP4, E8M0) or 16 (NVFP4, E4M3) elements of a row in the tile order
    qlora.h gives, and for NVFP4 a float scale, one or one per row."""
    codes: torch.Tensor                     # uint8 [rows * 16 * ceil(cols / 32)]
    scales: torch.Tensor                    # uint8, tiles of 512 bytes
    global_scale: torch.Tensor | None       # float32 [1] or [rows] (NVFP4)
    rows: int
    cols: int
    fmt: str = "mxfp4"                      # "mxfp4" or "nvfp4"

    @property
    def scale_per_row(self) -> bool:
        return self.global_scale is not None and self.rows != 1 and self.global_scale.numel() == self.rows

    @property
    def device(self):
        return self.codes.device

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.codes, self.scales, self.global_scale) if t is not None)

    def c_struct(self) -> _MxTensorC:
        """The C descriptor, after checking that the buffers hold what it describes."""
        c, s, g, rows, fmt = self.codes, self.scales, self.global_scale, self.rows, self.fmt
        if fmt not in MX_FORMATS:
            raise ValueError(f"fmt must be one of {sorted(MX_FORMATS)}")
        need_c, need_s = _mx_bytes(rows, self.cols, fmt)
        dev = c.device
        if not (c.dtype is torch.uint8 and s.dtype is torch.uint8 and c.is_contiguous() and s.is_contiguous()
                and c.is_cuda and dev == s.device):
            raise ValueError("codes and scales must be contiguous uint8 tensors on one CUDA device")
        if c.numel() < need_c or s.numel() < need_s:
            raise ValueError(f"a {rows}x{self.cols} {fmt} tensor needs {need_c} bytes of codes and {need_s} of scales")
        if (g is None) != (fmt == "mxfp4"):
            raise ValueError("global_scale belongs to nvfp4 and only to it")
        if g is None:
            return _MxTensorC(c.data_ptr(), s.data_ptr(), 0, rows, self.cols, 0, 0)
        n = g.numel()
        if not (g.dtype is torch.float32 and g.is_contiguous() and g.device == dev and (n == 1 or n == rows)):
            raise ValueError("global_scale must be a float32 tensor of 1 or `rows` elements on the codes' device")
        return _MxTensorC(c.data_ptr(), s.data_ptr(), g.data_ptr(), rows, self.cols, 1, 1 if n != 1 else 0)


def empty_mx(rows: int, cols: int, device, fmt: str = "mxfp4", per_row: bool = False) -> MXTensor:
    """An MXTensor with buffers for a [rows, cols] matrix."""
    if fmt not in MX_FORMATS:
        raise ValueError(f"fmt must be one of {sorted(MX_FORMATS)}")
    if per_row and fmt != "nvfp4":
        raise ValueError("a scale per row belongs to nvfp4")
    nc, ns = _mx_bytes(rows, cols, fmt)
    g = torch.empty(rows if per_row else 1, dtype=torch.float32, device=device) if fmt == "nvfp4" else None
    return MXTensor(torch.empty(nc, dtype=torch.uint8, device=device), torch.empty(ns, dtype=torch.uint8, device=device),
                    g, rows, cols, fmt)


def _on(device, where: str, fn, *args):
    """Call a C entry point with the tensors' device current and its current
    stream as the last argument."""
    i = device.index
    if torch.cuda.current_device() == i:
        status = fn(*args, _raw_stream(i))
    else:
        with torch.cuda.device(i):
            status = fn(*args, _raw_stream(i))
    if status != 0:
        raise QloraError(status, where)


# The current stream's handle of a device: torch's own getter where this torch has it,
# which builds no Stream object (2 us a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def qlora_mx_sizes(rows: int, cols: int, fmt: str = "mxfp4", per_row: bool = False) -> dict:
    """Buffer sizes in bytes of a microscaled matrix."""
    v = [ctypes.c_size_t() for _ in range(4)]
    _check(_lib.qlora_mx_sizes(rows, cols, MX_FORMATS[fmt], int(per_row), *[ctypes.byref(x) for x in v]), "qlora_mx_sizes")
    return dict(codes=v[0].value, scales=v[1].value, global_scale=v[2].value, workspace=v[3].value)


@functools.lru_cache(maxsize=4096)
def _mx_quant_workspace(rows: int, cols: int) -> int:
    """Work-buffer bytes of an NVFP4 quantisation with one global scale."""
    return qlora_mx_sizes(rows, cols, "nvfp4")["workspace"]


def qlora_mx_quantize(W: torch.Tensor, fmt: str = "mxfp4", transpose: bool = False, per_row: bool = False,
                      out: MXTensor | None = None, workspace: torch.Tensor | None = None) -> MXTensor:
    """Quantise a bf16 [rows, cols] matrix along its rows, or with `transpose`
    its transpose (the weight operand of qlora_mx_linear_bwd).  `per_row` gives
    an NVFP4 matrix one global scale per row instead of one in all; `out`, when
    given, fixes the format and the form."""
    _need_bf16_cuda("W", W)
    if W.dim() != 2:
        raise ValueError("W must be a matrix")
    rows, cols = (W.shape[1], W.shape[0]) if transpose else (W.shape[0], W.shape[1])
    if out is None:
        out = empty_mx(rows, cols, W.device, fmt, per_row)
    elif (out.rows, out.cols) != (rows, cols) or out.device != W.device:
        raise ValueError(f"out describes {out.rows}x{out.cols} on {out.device}, the result is {rows}x{cols} on {W.device}")
    if rows == 0 or cols == 0:
        return out
    c = out.c_struct()
    if workspace is not None:
        _mx_workspace(workspace, 0, W.device)
    elif out.fmt == "nvfp4" and not out.scale_per_row and _mx_quant_workspace(rows, cols):
        workspace = torch.empty(_mx_quant_workspace(rows, cols), dtype=torch.uint8, device=W.device)
    _on(W.device, "qlora_mx_quantize", _lib.qlora_mx_quantize, W.data_ptr(), int(transpose), c, _addr(workspace),
        _size(workspace))
    return out


def qlora_mx_dequantize(q: MXTensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """The values of a microscaled matrix as a bf16 [rows, cols] tensor."""
    if out is None:
        out = torch.empty(q.rows, q.cols, dtype=torch.bfloat16, device=q.device)
    else:
        _need_bf16_cuda("out", out)
        if out.shape != (q.rows, q.cols) or out.device != q.device:
            raise ValueError(f"out must be a {q.rows}x{q.cols} tensor on {q.device}")
    if q.rows == 0 or q.cols == 0:
        return out
    _on(q.device, "qlora_mx_dequantize", _lib.qlora_mx_dequantize, q.c_struct(), out.data_ptr())
    return out


def _addr(t):
    return None if t is None else t.data_ptr()


def _size(t) -> int:
    """Bytes of a work buffer (0 for none)."""
    return 0 if t is None else t.numel() * t.element_size()


@functools.lru_cache(maxsize=4096)
def qlora_mx_linear_workspace_size(rows: int, cols: int, fmt: str, m: int, r: int = 0) -> tuple:
    """(forward, backward) work-buffer bytes of a layer W [rows, cols]; r = 0: no adapter."""
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    _check(_lib.qlora_mx_linear_workspace_size(rows, cols, MX_FORMATS[fmt], m, r, f, b), "qlora_mx_linear_workspace_size")
    return f.value, b.value


def _need(name: str, t: torch.Tensor, dtype, shape: tuple, device):
    if not (t.dtype == dtype and t.shape == shape and t.device == device and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, "
                         f"not {t.dtype} {tuple(t.shape)} on {t.device}")


def _mx_workspace(workspace, need: int, device):
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return workspace


def qlora_mx_linear_fwd(q: MXTensor, X: torch.Tensor, A: torch.Tensor | None = None, B: torch.Tensor | None = None,
                        s: float = 0.0, save_xa: bool = True, Y: torch.Tensor | None = None,
                        XA: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """Y = deq(q(X)) deq(W)^T [+ s (X A^T) B^T] over a microscaled weight W
    [rows, cols]; X is quantised in W's format.  Without an adapter (A and B
    None) any sizes are taken.  Returns (Y bf16, X A^T fp32 or None)."""
    c, dev = q.c_struct(), q.device
    m = X.shape[0]
    _need("X", X, torch.bfloat16, (m, q.cols), dev)
    r = 0
    if (A is None) != (B is None):
        raise ValueError("A and B come together")
    if A is not None:
        r = A.shape[0]
        _need("A", A, torch.bfloat16, (r, q.cols), dev)
        _need("B", B, torch.bfloat16, (q.rows, r), dev)
    if Y is None:
        Y = torch.empty(m, q.rows, dtype=torch.bfloat16, device=dev)
    else:
        _need("Y", Y, torch.bfloat16, (m, q.rows), dev)
    if not (r and save_xa):
        XA = None
    elif XA is None:
        XA = torch.empty(m, r, dtype=torch.float32, device=dev)
    else:
        _need("XA", XA, torch.float32, (m, r), dev)
    workspace = _mx_workspace(workspace, qlora_mx_linear_workspace_size(q.rows, q.cols, q.fmt, m, r)[0], dev)
    _on(dev, "qlora_mx_linear_fwd", _lib.qlora_mx_linear_fwd, c, X.data_ptr(), m, _addr(A), _addr(B), r, float(s),
        Y.data_ptr(), _addr(XA), workspace.data_ptr(), _size(workspace))
    return Y, XA


def qlora_mx_linear_bwd(qT: MXTensor, dY: torch.Tensor, X: torch.Tensor | None = None, A: torch.Tensor | None = None,
                        B: torch.Tensor | None = None, s: float = 0.0, XA: torch.Tensor | None = None,
                        need_dx: bool = True, dX: torch.Tensor | None = None, dA: torch.Tensor | None = None,
                        dB: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """Backward of qlora_mx_linear_fwd.  qT holds the layer's weight transposed,
    [cols, rows] (qlora_mx_quantize(W, transpose=True)).  Returns (dX bf16 or
    None, dA fp32, dB fp32); without an adapter dA and dB are None."""
    c, dev = qT.c_struct(), qT.device
    rows, cols, m, r = qT.cols, qT.rows, dY.shape[0], 0
    _need("dY", dY, torch.bfloat16, (m, rows), dev)
    if (A is None) != (B is None):
        raise ValueError("A and B come together")
    if A is not None:
        r = A.shape[0]
        if X is None:
            raise ValueError("the adapter's gradients need X")
        _need("X", X, torch.bfloat16, (m, cols), dev)
        _need("A", A, torch.bfloat16, (r, cols), dev)
        _need("B", B, torch.bfloat16, (rows, r), dev)
        if XA is not None:
            _need("XA", XA, torch.float32, (m, r), dev)
        if dA is None:
            dA = torch.empty(r, cols, dtype=torch.float32, device=dev)
        else:
            _need("dA", dA, torch.float32, (r, cols), dev)
        if dB is None:
            dB = torch.empty(rows, r, dtype=torch.float32, device=dev)
        else:
            _need("dB", dB, torch.float32, (rows, r), dev)
    else:
        X = XA = dA = dB = None
    if not need_dx:
        dX = None
    elif dX is None:
        dX = torch.empty(m, cols, dtype=torch.bfloat16, device=dev)
    else:
        _need("dX", dX, torch.bfloat16, (m, cols), dev)
    workspace = _mx_workspace(workspace, qlora_mx_linear_workspace_size(rows, cols, qT.fmt, m, r)[1], dev)
    _on(dev, "qlora_mx_linear_bwd", _lib.qlora_mx_linear_bwd, c, _addr(X), dY.data_ptr(), m, _addr(A), _addr(B), r,
        float(s), _addr(XA), _addr(dX), _addr(dA), _addr(dB), workspace.data_ptr(), _size(workspace))
    return dX, dA, dB


def qlora_selftest_mx_form(rows: int, cols: int, fmt: str, m: int, r: int = 0, backward: bool = False,
                           num_sms: int = 148) -> tuple:
    """("few", "stream" or "pair", token tile): the kernel that multiplies in a
    forward or a backward of a layer W [rows, cols] (for tests)."""
    form, tile = ctypes.c_int32(), ctypes.c_int32()
    _check(_lib.qlora_selftest_mx_form(rows, cols, MX_FORMATS[fmt], m, r, int(backward), num_sms, form, tile),
           "qlora_selftest_mx_form")
    return ("few", "stream", "pair")[form.value], tile.value


@functools.lru_cache(maxsize=4096)
def qlora_mx_moe_workspace_size(experts: int, hidden: int, inner: int, m: int, top_k: int) -> int:
    b = ctypes.c_size_t()
    _check(_lib.qlora_mx_moe_workspace_size(experts, hidden, inner, m, top_k, b), "qlora_mx_moe_workspace_size")
    return b.value


def qlora_mx_moe_fwd(W13: MXTensor, W2: MXTensor, router: torch.Tensor, X: torch.Tensor, top_k: int,
                     Y: torch.Tensor | None = None, ids: torch.Tensor | None = None, probs: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None):
    """A mixture-of-experts layer for at most 16 tokens: W13 stacks the experts'
    gate and up rows [experts * 2 inner, hidden], W2 their down rows
    [experts * hidden, inner], both MXFP4; router [experts, hidden] bf16.
    Returns (Y bf16 [m, hidden], ids int32 [m, top_k], probs fp32 [m, top_k])."""
    c13, c2, dev = W13.c_struct(), W2.c_struct(), W13.device
    if W2.device != dev:
        raise ValueError(f"W2 is on {W2.device}, W13 on {dev}")
    m, experts, hidden = X.shape[0], router.shape[0], W13.cols
    _need("X", X, torch.bfloat16, (m, hidden), dev)
    _need("router", router, torch.bfloat16, (experts, hidden), dev)
    if W13.rows != experts * 2 * W2.cols or W2.rows != experts * hidden:
        raise ValueError(f"{experts} experts of hidden {hidden} and inner {W2.cols}: W13 must have {experts * 2 * W2.cols} rows "
                         f"and W2 {experts * hidden}, not {W13.rows} and {W2.rows}")
    if Y is None:
        Y = torch.empty(m, hidden, dtype=torch.bfloat16, device=dev)
    else:
        _need("Y", Y, torch.bfloat16, (m, hidden), dev)
    if ids is None:
        ids = torch.empty(m, max(top_k, 0), dtype=torch.int32, device=dev)
    else:
        _need("ids", ids, torch.int32, (m, top_k), dev)
    if probs is None:
        probs = torch.empty(m, max(top_k, 0), dtype=torch.float32, device=dev)
    else:
        _need("probs", probs, torch.float32, (m, top_k), dev)
    workspace = _mx_workspace(workspace, qlora_mx_moe_workspace_size(experts, hidden, W2.cols, m, top_k), dev)
    _on(dev, "qlora_mx_moe_fwd", _lib.qlora_mx_moe_fwd, c13, c2, router.data_ptr(), experts, X.data_ptr(), m, top_k,
        Y.data_ptr(), ids.data_ptr(), probs.data_ptr(), workspace.data_ptr(), _size(workspace))
    return Y, ids, probs
