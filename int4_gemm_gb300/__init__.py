"""Python binding of the q4gemm C ABI (``include/q4gemm.h``).

Argument marshalling only: tensors are passed by ``data_ptr()`` together with
torch's current CUDA stream, and every step runs in the library's kernels.
PyTorch provides device memory (outputs and workspaces are torch tensors
allocated here, on the caller's side of the ABI) and streams.  There is no
fallback: if ``libq4gemm.so`` is missing or a call fails, an exception is
raised.

A call runs on the current stream, or on ``stream``, whose memory its own outputs
and workspaces then are: work that is pending elsewhere does not touch them, and
the current stream may read them (after waiting for ``stream``) and let them go.
Ordering ``stream`` with the inputs, and with an ``out`` or ``ws`` that is given,
is the caller's part, as under ``torch.cuda.stream``.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional, Union

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libq4gemm.so")

Q4_OK = 0
F32, BF16, F16 = 0, 1, 2
ROWMAJOR, MMA = 0, 1
OP_QUANTIZE_NVFP4, OP_GEMM_W4A4_NVFP4, OP_GEMM_W4A4_MXFP4, OP_GEMM_W4A16_INT4 = 0, 1, 2, 3
OP_GROUPED_GEMM_MOE, OP_GEMM_W4A16_NVFP4, OP_GEMM_W4A16_MXFP4 = 4, 5, 6
OP_GEMM_FP8_BLOCKWISE, OP_GEMM_W4A8 = 7, 8
OP_GEMM_W4A4_MXFP4_FUSED = 9
OP_MOE_SORT, OP_GROUPED_WGRAD_FP8 = 10, 11

_DTYPE = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
_LAYOUT = {"rowmajor": ROWMAJOR, "mma": MMA}
_NORMALIZE = {"topk": 0, "all": 1}  # q4_route_normalize: softmax over the chosen / over all logits
_ROUNDING = {"pages": 0, "rne": 1}  # q4_rounding: E2M1 ties to the smaller magnitude / to even

_lib: Optional[ctypes.CDLL] = None


class Q4Error(RuntimeError):
    def __init__(self, fn: str, status: int):
        msg = _lib.q4_status_string(status).decode() if _lib is not None else str(status)
        super().__init__(f"{fn} failed: {msg} ({status})")
        self.status = status


class _Operand(ctypes.Structure):
    _fields_ = [("raw", ctypes.c_void_p), ("raw_dtype", ctypes.c_int),
                ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("scale_layout", ctypes.c_int), ("tensor_scale", ctypes.c_void_p)]


def _sig(lib, name, restype, *argtypes):
    f = getattr(lib, name)
    f.restype = restype
    f.argtypes = list(argtypes)


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the library (built by ``__graft_entry__.build()`` or
    ``python -m int4_gemm_gb300.build``).  Raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m int4_gemm_gb300.build`")
    lib = ctypes.CDLL(path)
    P, I, I64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    _sig(lib, "q4_workspace_size", SZ, I, I64, I64, I64)
    _sig(lib, "q4_workspace_size_moe", SZ, I64, I64, I64, I, I64)
    _sig(lib, "q4_workspace_size_wgrad", SZ, I64, I64, I64, I)
    _sig(lib, "q4_mma_scales_bytes", SZ, I64, I64)
    _sig(lib, "quantize_nvfp4", I, P, I, I64, I64, P, P, I, P, P, SZ, P)
    _sig(lib, "quantize_mxfp4", I, P, I, I64, I64, P, P, I, P)
    _sig(lib, "quantize_nvfp4_ex", I, P, I, I64, I64, P, P, I, I, P, P, SZ, P)
    _sig(lib, "quantize_mxfp4_ex", I, P, I, I64, I64, P, P, I, I, P)
    _sig(lib, "quantize_int4_g128", I, P, I, I64, I64, P, P, P)
    _sig(lib, "q4_scales_to_mma", I, P, I64, I64, P, P)
    op = ctypes.POINTER(_Operand)
    _sig(lib, "gemm_w4a4_nvfp4", I, op, op, I64, I64, I64, P, I, P, SZ, P)
    _sig(lib, "gemm_w4a4_mxfp4", I, op, op, I64, I64, I64, P, I, P, SZ, P)
    _sig(lib, "gemm_w4a4_mxfp4_fused", I, P, I, op, I64, I64, I64, P, I, P, SZ, P)
    _sig(lib, "gemm_w4a16_int4", I, P, P, P, I64, I64, I64, P, P, SZ, P)
    _sig(lib, "gemm_w4a16_nvfp4", I, P, P, P, P, I64, I64, I64, P, P, SZ, P)
    _sig(lib, "gemm_w4a16_mxfp4", I, P, P, P, I64, I64, I64, P, P, SZ, P)
    _sig(lib, "grouped_gemm_moe", I, P, I64, I64, P, P, I64, I, op, I64, P, P, SZ, P)
    _sig(lib, "quantize_fp8_blockwise", I, P, I, I64, I64, I, P, P, P)
    _sig(lib, "gemm_fp8_blockwise", I, P, P, P, P, I64, I64, I64, P, I, P, SZ, P)
    _sig(lib, "w4a8_weight_scales", I, P, I64, I64, P, P)
    _sig(lib, "gemm_w4a8", I, P, P, P, P, I64, I64, I64, P, I, P, SZ, P)
    _sig(lib, "moe_route_topk", I, P, I, I64, I64, I64, I, I, P, P, P)
    _sig(lib, "moe_route_topk_backward", I, P, I, I64, I64, I64, I, I, P, P, P, P)
    _sig(lib, "moe_sort_tokens", I, P, I64, I, I, P, P, P, P, SZ, P)
    _sig(lib, "moe_dispatch", I, P, I, I64, I64, I64, P, I, P, P)
    _sig(lib, "moe_dispatch_backward", I, P, I, I64, I64, I64, P, I, P, P)
    _sig(lib, "moe_combine", I, P, I, I64, I64, I64, P, P, I, P, P)
    _sig(lib, "moe_combine_backward", I, P, I, I64, I64, I64, P, I64, P, P, I, P, P, P)
    _sig(lib, "quantize_fp8_checkpoint", I, P, I, I64, I64, I64, P, P, P)
    _sig(lib, "swiglu_fp8", I, P, I, I64, I64, I64, P, P, P, P)
    _sig(lib, "swiglu_fp8_backward", I, P, I, I64, I64, I64, P, P, P, P)
    _sig(lib, "grouped_wgrad_fp8", I, P, I64, I64, I64, P, P, I64, I64, P, P, I, P, I, I, P, SZ, P)
    _sig(lib, "q4_sync_status", I, P)
    _sig(lib, "q4_status_string", ctypes.c_char_p, I)
    _sig(lib, "q4_set_wait_timeout_ms", I, I)
    _sig(lib, "q4_selftest_wait_timeout", I, P)
    _sig(lib, "q4_read_probe_sink_words", SZ)
    _sig(lib, "q4_read_probe", I, P, SZ, P, P)
    _sig(lib, "gemm_w4a4_nvfp4_noalloc", I, P, I, op, I64, I64, I64, P, I, P)
    _sig(lib, "q4_noalloc_scratch_bytes", SZ)
    _sig(lib, "q4_noalloc_required_bytes", SZ, I64, I64)
    _lib = lib
    return lib


def lib() -> ctypes.CDLL:
    return load()


def _check(fn: str, status: int):
    if status != Q4_OK:
        raise Q4Error(fn, status)


# The current stream's handle without building a Stream object (a few us per
# call otherwise); the public route where this build of torch lacks it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream=None) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(_device())
    return torch.cuda.current_stream().cuda_stream


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _cuda2d(x: torch.Tensor, name: str) -> torch.Tensor:
    if not x.is_cuda or x.dim() != 2 or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 2-D CUDA tensor")
    return x


def _new(shape, dtype: torch.dtype, device, stream=None, result: bool = True) -> torch.Tensor:
    """New memory for a call on ``stream``.  Recycled memory is safe on the stream
    that it is allocated for only (kernels of another may still be about to
    write it), so it is allocated for the call's; the current stream is recorded as
    a user of the results."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if result:
        t.record_stream(torch.cuda.current_stream(t.device))
    return t


def _given(t: torch.Tensor, stream) -> torch.Tensor:
    """The caller's tensor, not reused before ``stream`` is done with it."""
    if stream is not None:
        t.record_stream(stream)
    return t


def _out(out: Optional[torch.Tensor], M: int, N: int, dtype: torch.dtype, device, stream=None) -> torch.Tensor:
    """A new [M, N] output, or the caller's, checked against the call."""
    if out is None:
        return _new((M, N), dtype, device, stream)
    if (tuple(out.shape) != (M, N) or out.dtype != dtype or out.device != torch.device(device)
            or not out.is_contiguous()):
        raise ValueError(f"out must be a contiguous {dtype} tensor of shape ({M}, {N}) on {device}")
    return _given(out, stream)


def _empty(nbytes: int, device, stream=None) -> torch.Tensor:
    """A workspace."""
    return _new(max(int(nbytes), 0), torch.uint8, device, stream, result=False)


def workspace(op: int, M: int, N: int, K: int, device, stream=None) -> torch.Tensor:
    n = lib().q4_workspace_size(op, M, N, K)
    ws = _empty(max(n, 256), device, stream)
    if op == OP_GEMM_W4A4_MXFP4_FUSED:  # the grid gate's counters start at zero
        with torch.cuda.stream(stream):  # None: the current one
            ws[:256].zero_()
    return ws


def mma_scales_bytes(rows: int, nsf: int) -> int:
    return int(lib().q4_mma_scales_bytes(rows, nsf))


# --------------------------------------------------------------------------- quantizers

def quantize_nvfp4(x: torch.Tensor, scale_layout: str = "rowmajor", rounding: str = "pages",
                   stream=None):
    """-> (codes u8 [rows, K/2], scales u8, tensor_scale f32 [1]).
    rounding: "pages" (E2M1 ties to the smaller magnitude) or "rne"."""
    _cuda2d(x, "x")
    rows, K = x.shape
    dev = x.device
    codes = _new((rows, K // 2), torch.uint8, dev, stream)
    lay = _LAYOUT[scale_layout]
    if lay == ROWMAJOR:
        scales = _new((rows, K // 16), torch.uint8, dev, stream)
    else:
        scales = _new(mma_scales_bytes(rows, K // 16), torch.uint8, dev, stream)
    ts = _new(1, torch.float32, dev, stream)
    ws = workspace(OP_QUANTIZE_NVFP4, rows, 0, K, dev, stream)
    _check("quantize_nvfp4", lib().quantize_nvfp4_ex(
        x.data_ptr(), _DTYPE[x.dtype], rows, K, codes.data_ptr(), scales.data_ptr(), lay,
        _ROUNDING[rounding], ts.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream)))
    return codes, scales, ts


def quantize_mxfp4(x: torch.Tensor, scale_layout: str = "rowmajor", rounding: str = "pages",
                   stream=None):
    """-> (codes u8 [rows, K/2], scales u8).
    rounding: "pages" (E2M1 ties to the smaller magnitude) or "rne"."""
    _cuda2d(x, "x")
    rows, K = x.shape
    dev = x.device
    codes = _new((rows, K // 2), torch.uint8, dev, stream)
    lay = _LAYOUT[scale_layout]
    if lay == ROWMAJOR:
        scales = _new((rows, K // 32), torch.uint8, dev, stream)
    else:
        scales = _new(mma_scales_bytes(rows, K // 32), torch.uint8, dev, stream)
    _check("quantize_mxfp4", lib().quantize_mxfp4_ex(
        x.data_ptr(), _DTYPE[x.dtype], rows, K, codes.data_ptr(), scales.data_ptr(), lay,
        _ROUNDING[rounding], _stream(stream)))
    return codes, scales


def quantize_int4_g128(x: torch.Tensor, stream=None):
    """-> (codes u8 [rows, K/2], scales int16 [rows, K/128] holding FP16 bits)."""
    _cuda2d(x, "x")
    rows, K = x.shape
    codes = _new((rows, K // 2), torch.uint8, x.device, stream)
    scales = _new((rows, K // 128), torch.int16, x.device, stream)
    _check("quantize_int4_g128", lib().quantize_int4_g128(
        x.data_ptr(), _DTYPE[x.dtype], rows, K, codes.data_ptr(), scales.data_ptr(),
        _stream(stream)))
    return codes, scales


def scales_to_mma(src: torch.Tensor, stream=None) -> torch.Tensor:
    _cuda2d(src, "src")
    rows, nsf = src.shape
    dst = _new(mma_scales_bytes(rows, nsf), torch.uint8, src.device, stream)
    _check("q4_scales_to_mma", lib().q4_scales_to_mma(src.data_ptr(), rows, nsf, dst.data_ptr(),
                                                      _stream(stream)))
    return dst


# --------------------------------------------------------------------------- GEMMs

@dataclass
class Fp4Operand:
    """A quantized FP4 operand as returned by quantize_nvfp4 / quantize_mxfp4."""
    codes: torch.Tensor
    scales: torch.Tensor
    scale_layout: str = "rowmajor"
    tensor_scale: Optional[torch.Tensor] = None


def _operand(x: Union[torch.Tensor, Fp4Operand], K: int) -> tuple[_Operand, int]:
    if isinstance(x, Fp4Operand):
        _cuda2d(x.codes, "operand codes")
        if x.codes.shape[1] * 2 != K:
            raise ValueError(f"operand codes hold K = {x.codes.shape[1] * 2}, not {K}")
        return _Operand(None, 0, x.codes.data_ptr(), x.scales.data_ptr(), _LAYOUT[x.scale_layout],
                        _ptr(x.tensor_scale)), x.codes.shape[0]
    _cuda2d(x, "operand")
    if x.shape[1] != K:
        raise ValueError(f"operand has K = {x.shape[1]}, not {K}")
    return _Operand(x.data_ptr(), _DTYPE[x.dtype], None, None, 0, None), x.shape[0]


def _gemm_fp4(fn: str, op: int, A, B, K: int, out_dtype: torch.dtype, stream=None, ws=None,
              out=None) -> torch.Tensor:
    a, M = _operand(A, K)
    b, N = _operand(B, K)
    dev = (A.codes if isinstance(A, Fp4Operand) else A).device
    C = _out(out, M, N, out_dtype, dev, stream)
    if ws is None:
        ws = workspace(op, M, N, K, dev, stream)
    _check(fn, getattr(lib(), fn)(ctypes.byref(a), ctypes.byref(b), M, N, K, C.data_ptr(),
                                  _DTYPE[out_dtype], ws.data_ptr(), ws.numel(), _stream(stream)))
    return C


def gemm_w4a4_nvfp4(A, B, K: int, out_dtype=torch.bfloat16, stream=None, ws=None,
                    out=None) -> torch.Tensor:
    """C = A_hat . B_hat^T; A and B are raw tensors (quantized on the fly) or
    Fp4Operand.  ``ws`` (from :func:`workspace`) and ``out`` may be given to
    keep allocations out of a CUDA-graph capture."""
    return _gemm_fp4("gemm_w4a4_nvfp4", OP_GEMM_W4A4_NVFP4, A, B, K, out_dtype, stream, ws, out)


def gemm_w4a4_mxfp4(A, B, K: int, out_dtype=torch.bfloat16, stream=None, ws=None,
                    out=None) -> torch.Tensor:
    return _gemm_fp4("gemm_w4a4_mxfp4", OP_GEMM_W4A4_MXFP4, A, B, K, out_dtype, stream, ws, out)


def gemm_w4a4_mxfp4_fused(A: torch.Tensor, B, K: int, out_dtype=torch.bfloat16, stream=None,
                          ws=None, out=None) -> torch.Tensor:
    """gemm_w4a4_mxfp4 of a raw A in one launch: the GEMM quantizes A in its
    prologue.  ``ws`` must come from ``workspace(OP_GEMM_W4A4_MXFP4_FUSED,
    ...)`` (its first 256 bytes are the gate's counters, zero before the first
    call; each call leaves them zero)."""
    _cuda2d(A, "A")
    if A.shape[1] != K:
        raise ValueError(f"A has K = {A.shape[1]}, not {K}")
    b, N = _operand(B, K)
    M = A.shape[0]
    C = _out(out, M, N, out_dtype, A.device, stream)
    if ws is None:
        ws = workspace(OP_GEMM_W4A4_MXFP4_FUSED, M, N, K, A.device, stream)
    _check("gemm_w4a4_mxfp4_fused",
           lib().gemm_w4a4_mxfp4_fused(A.data_ptr(), _DTYPE[A.dtype], ctypes.byref(b), M, N, K,
                                       C.data_ptr(), _DTYPE[out_dtype], ws.data_ptr(), ws.numel(),
                                       _stream(stream)))
    return C


def gemm_w4a4_nvfp4_noalloc(A: torch.Tensor, B: Fp4Operand, K: int, out_dtype=torch.bfloat16,
                            out=None, stream=None) -> torch.Tensor:
    """gemm_w4a4_nvfp4 with raw activations for callers that cannot provide a
    workspace: the quantized activations go to the library's fixed 16 MiB
    per-GPU scratch array (see include/q4gemm.h).  B must carry MMA-layout
    scales.  Calls that overlap on the GPU share that scratch and race."""
    if not isinstance(A, torch.Tensor):
        raise ValueError("A must be the raw activation tensor")
    _, M = _operand(A, K)
    b, N = _operand(B, K)
    C = _out(out, M, N, out_dtype, A.device, stream)
    _check("gemm_w4a4_nvfp4_noalloc", lib().gemm_w4a4_nvfp4_noalloc(
        A.data_ptr(), _DTYPE[A.dtype], ctypes.byref(b), M, N, K, C.data_ptr(), _DTYPE[out_dtype],
        _stream(stream)))
    return C


def gemm_w4a16_int4(A: torch.Tensor, Wq: torch.Tensor, Ws: torch.Tensor, out=None,
                    stream=None, ws=None) -> torch.Tensor:
    """C [M, N] bf16 = A [M, K] bf16 . dequant(Wq, Ws)^T.  ``ws``: optional
    workspace (q4_workspace_size gives 0 for this call today)."""
    _cuda2d(A, "A")
    M, K = A.shape
    N = Wq.shape[0]
    C = _out(out, M, N, torch.bfloat16, A.device, stream)
    _check("gemm_w4a16_int4", lib().gemm_w4a16_int4(A.data_ptr(), Wq.data_ptr(), Ws.data_ptr(), M,
                                                     N, K, C.data_ptr(), _ptr(ws), 0 if ws is None else ws.numel(),
                                                     _stream(stream)))
    return C


def gemm_w4a16_nvfp4(A: torch.Tensor, Wq: torch.Tensor, Ws: torch.Tensor, Wg: torch.Tensor,
                     out=None, stream=None, ws=None) -> torch.Tensor:
    """C [M, N] bf16 = A [M, K] bf16 . dequant(W)^T, W NVFP4: codes [N, K/2],
    row-major E4M3 scales [N, K/16], tensor scale Wg (one float32)."""
    _cuda2d(A, "A")
    M, K = A.shape
    N = Wq.shape[0]
    C = _out(out, M, N, torch.bfloat16, A.device, stream)
    _check("gemm_w4a16_nvfp4", lib().gemm_w4a16_nvfp4(A.data_ptr(), Wq.data_ptr(), Ws.data_ptr(),
                                                       Wg.data_ptr(), M, N, K, C.data_ptr(),
                                                       _ptr(ws), 0 if ws is None else ws.numel(),
                                                       _stream(stream)))
    return C


def gemm_w4a16_mxfp4(A: torch.Tensor, Wq: torch.Tensor, Ws: torch.Tensor, out=None,
                     stream=None, ws=None) -> torch.Tensor:
    """C [M, N] bf16 = A [M, K] bf16 . dequant(W)^T, W MXFP4: codes [N, K/2],
    row-major E8M0 scales [N, K/32]."""
    _cuda2d(A, "A")
    M, K = A.shape
    N = Wq.shape[0]
    C = _out(out, M, N, torch.bfloat16, A.device, stream)
    _check("gemm_w4a16_mxfp4", lib().gemm_w4a16_mxfp4(A.data_ptr(), Wq.data_ptr(), Ws.data_ptr(),
                                                       M, N, K, C.data_ptr(), _ptr(ws),
                                                       0 if ws is None else ws.numel(),
                                                       _stream(stream)))
    return C


def quantize_fp8_blockwise(x: torch.Tensor, block_rows: int, codes=None, scales=None,
                           stream=None):
    """FP8 (E4M3) blockwise quantization of x [rows, K] (f32 / bf16 / f16):
    block_rows 128 for weights (128 x 128 blocks), 1 for activations (1 x 128).
    -> (codes u8 [rows, K], scales float32 [rows / block_rows, K / 128])."""
    _cuda2d(x, "x")
    rows, K = x.shape
    if codes is None:
        codes = _new((rows, K), torch.uint8, x.device, stream)
    if scales is None:
        scales = _new((rows // max(block_rows, 1), K // 128), torch.float32, x.device, stream)
    _check("quantize_fp8_blockwise", lib().quantize_fp8_blockwise(
        x.data_ptr(), _DTYPE[x.dtype], rows, K, block_rows, codes.data_ptr(), scales.data_ptr(),
        _stream(stream)))
    return codes, scales


def gemm_fp8_blockwise(qa: torch.Tensor, sa: torch.Tensor, qb: torch.Tensor, sb: torch.Tensor,
                       out_dtype=torch.bfloat16, out=None, stream=None) -> torch.Tensor:
    """C [M, N] = sum over 128-wide K blocks of sa * sb * (qa . qb^T): qa E4M3
    [M, K] with sa [M, K/128], qb E4M3 [N, K] with sb [N/128, K/128]."""
    _cuda2d(qa, "qa")
    M, K = qa.shape
    N = qb.shape[0]
    C = _out(out, M, N, out_dtype if out is None else out.dtype, qa.device, stream)
    _check("gemm_fp8_blockwise", lib().gemm_fp8_blockwise(
        qa.data_ptr(), sa.data_ptr(), qb.data_ptr(), sb.data_ptr(), M, N, K, C.data_ptr(),
        _DTYPE[C.dtype], None, 0, _stream(stream)))
    return C


def w4a8_weight_scales(w_scales: torch.Tensor, stream=None) -> torch.Tensor:
    """FP16 INT4 group scales [N, K/128] (as quantize_int4_g128 returns them,
    int16 bits) -> float32 [K/128, N], the layout gemm_w4a8 reads."""
    _cuda2d(w_scales, "w_scales")
    N, KB = w_scales.shape
    out = _new((KB, N), torch.float32, w_scales.device, stream)
    _check("w4a8_weight_scales", lib().w4a8_weight_scales(
        w_scales.data_ptr(), N, KB * 128, out.data_ptr(), _stream(stream)))
    return out


def gemm_w4a8(qa: torch.Tensor, sa: torch.Tensor, w_codes: torch.Tensor, w_scales_kn: torch.Tensor,
              out_dtype=torch.bfloat16, out=None, stream=None) -> torch.Tensor:
    """C [M, N] = sum over 128-wide K blocks of sa * s16 * (qa . q^T): qa E4M3
    [M, K] with sa [M, K/128]; INT4 codes [N, K/2] with w4a8_weight_scales'
    float32 [K/128, N]."""
    _cuda2d(qa, "qa")
    M, K = qa.shape
    N = w_codes.shape[0]
    C = _out(out, M, N, out_dtype if out is None else out.dtype, qa.device, stream)
    _check("gemm_w4a8", lib().gemm_w4a8(
        qa.data_ptr(), sa.data_ptr(), w_codes.data_ptr(), w_scales_kn.data_ptr(), M, N, K,
        C.data_ptr(), _DTYPE[C.dtype], None, 0, _stream(stream)))
    return C


def moe_workspace(T: int, N: int, K: int, E: int, R: int, device,
                  w_scale_layout: str = "mma", stream=None) -> torch.Tensor:
    n = int(lib().q4_workspace_size_moe(T, N, K, E, R))
    if w_scale_layout == "rowmajor":  # room for the weight scales in the tensor-core layout
        n += E * mma_scales_bytes(N, K // 16)
    return _empty(max(n, 256), device, stream)


def grouped_gemm_moe(tokens: torch.Tensor, expert_offsets: torch.Tensor, row_token: torch.Tensor,
                     w_codes: torch.Tensor, w_scales: torch.Tensor, w_tensor_scales: torch.Tensor,
                     N: int, ws: Optional[torch.Tensor] = None, out=None, stream=None,
                     w_scale_layout: str = "mma") -> torch.Tensor:
    """C [R, N] bf16: routed rows times their expert's NVFP4 weights; rows from
    expert_offsets[E] on (dropped slots) are zero.
    w_codes [E, N, K/2]; w_scales: E stacked MMA-layout scale tensors, or
    [E, N, K/16] row-major bytes with ``w_scale_layout="rowmajor"``;
    w_tensor_scales [E] float32; expert_offsets [E+1] / row_token [R] int32."""
    _cuda2d(tokens, "tokens")
    T, K = tokens.shape
    E = expert_offsets.numel() - 1
    R = row_token.numel()
    C = _out(out, R, N, torch.bfloat16, tokens.device, stream)
    if ws is None:
        ws = moe_workspace(T, N, K, E, R, tokens.device, w_scale_layout, stream)
    w = _Operand(None, 0, w_codes.data_ptr(), w_scales.data_ptr(), _LAYOUT[w_scale_layout],
                 w_tensor_scales.data_ptr())
    _check("grouped_gemm_moe", lib().grouped_gemm_moe(
        tokens.data_ptr(), T, K, expert_offsets.data_ptr(), row_token.data_ptr(), R, E,
        ctypes.byref(w), N, C.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream)))
    return C


# --------------------------------------------------------------------------- routed experts

def _pitched(x: torch.Tensor, name: str) -> int:
    """The row pitch (at least the width) of a 2-D CUDA matrix whose rows are
    contiguous and do not overlap."""
    if not x.is_cuda or x.dtype not in _DTYPE or x.dim() != 2:
        raise ValueError(f"{name} must be a 2-D CUDA tensor of float32, bfloat16 or float16")
    (rows, cols), (pitch, step) = x.shape, x.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{name} must have contiguous rows")
    if rows <= 1 or cols == 0:  # no row has a next one, or no row has an element
        return cols
    if pitch < cols:
        raise ValueError(f"{name} has overlapping rows")
    return pitch


def _exact(t: torch.Tensor, name: str, shape, dtype: torch.dtype, device) -> torch.Tensor:
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.device == device:
        return t
    raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape} on {device}")


def _slots(slot_row: torch.Tensor, T: int, device) -> int:
    shape = slot_row.shape
    if len(shape) != 2:
        raise ValueError("slot_row must be a [T, top_k] tensor")
    k = shape[1]
    _exact(slot_row, "slot_row", (T, k), torch.int32, device)
    return k


def moe_route_topk(logits: torch.Tensor, top_k: int, normalize: str = "topk", stream=None):
    """The top_k experts of every token and their softmax weights.
    logits [T, E] (f32 / bf16 / f16, any row pitch; -inf masks an expert) ->
    (ids int32 [T, top_k], weights float32 [T, top_k]).  normalize: "topk"
    (softmax over the chosen logits) or "all" (over every logit)."""
    ld = _pitched(logits, "logits")
    T, E = logits.shape
    if abs(top_k) >= 1 << 31:
        raise ValueError("top_k must fit in 32 bits")
    slots = (T, top_k if 0 < top_k <= E else 0)  # none: refused below
    ids = _new(slots, torch.int32, logits.device, stream)
    weights = _new(slots, torch.float32, logits.device, stream)
    _check("moe_route_topk", lib().moe_route_topk(
        logits.data_ptr(), _DTYPE[logits.dtype], T, E, ld, top_k, _NORMALIZE[normalize],
        ids.data_ptr(), weights.data_ptr(), _stream(stream)))
    return ids, weights


def moe_route_topk_backward(logits: torch.Tensor, ids: torch.Tensor, d_weights: torch.Tensor,
                            normalize: str = "topk", stream=None) -> torch.Tensor:
    """d_logits [T, E] (logits' dtype) of moe_route_topk from d_weights float32 [T, top_k]."""
    ld = _pitched(logits, "logits")
    T, E = logits.shape
    if ids.dim() != 2:
        raise ValueError("ids must be a [T, top_k] tensor")
    k = ids.shape[1]
    _exact(ids, "ids", (T, k), torch.int32, logits.device)
    _exact(d_weights, "d_weights", (T, k), torch.float32, logits.device)
    d = _new((T, E), logits.dtype, logits.device, stream)
    _check("moe_route_topk_backward", lib().moe_route_topk_backward(
        logits.data_ptr(), _DTYPE[logits.dtype], T, E, ld, k, _NORMALIZE[normalize],
        ids.data_ptr(), d_weights.data_ptr(), d.data_ptr(), _stream(stream)))
    return d


def moe_sort_tokens(ids: torch.Tensor, E: int, ws: Optional[torch.Tensor] = None, stream=None):
    """Slots of ids int32 [T, top_k] sorted by expert -> (expert_offsets int32
    [E+1], row_token int32 [T*top_k], slot_row int32 [T, top_k]): the first two
    are grouped_gemm_moe's; slot_row holds every slot's row, or ~row where the
    id is outside [0, E) (dropped; those rows come last).  ``ws`` from
    ``workspace(OP_MOE_SORT, T * top_k, E, 0, device)``."""
    if not ids.is_cuda or ids.dim() != 2:
        raise ValueError("ids must be a [T, top_k] CUDA tensor")
    T, k = ids.shape
    dev = ids.device
    _exact(ids, "ids", (T, k), torch.int32, dev)
    if not 0 < E < 1 << 31:
        raise ValueError("E must be positive and fit in 32 bits")
    offsets = _new(E + 1, torch.int32, dev, stream)
    row_token = _new(T * k, torch.int32, dev, stream)
    slot_row = _new((T, k), torch.int32, dev, stream)
    L = lib()
    if ws is None:
        n = L.q4_workspace_size(OP_MOE_SORT, T * k, E, 0)
        ws = _empty(n, dev, stream) if n else None
    else:
        _given(ws, stream)
    _check("moe_sort_tokens", L.moe_sort_tokens(
        ids.data_ptr(), T, k, E, offsets.data_ptr(), row_token.data_ptr(), slot_row.data_ptr(),
        _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)))
    return offsets, row_token, slot_row


def moe_dispatch(x: torch.Tensor, slot_row: torch.Tensor, out=None, stream=None) -> torch.Tensor:
    """rows [T*top_k, H]: x [T, H] copied to every slot's row; rows of dropped slots are zero."""
    ld = _pitched(x, "x")
    T, H = x.shape
    k = _slots(slot_row, T, x.device)
    rows = _out(out, T * k, H, x.dtype, x.device, stream)
    _check("moe_dispatch", lib().moe_dispatch(x.data_ptr(), _DTYPE[x.dtype], T, H, ld,
                                              slot_row.data_ptr(), k, rows.data_ptr(), _stream(stream)))
    return rows


def moe_dispatch_backward(d_rows: torch.Tensor, slot_row: torch.Tensor, out=None,
                          stream=None) -> torch.Tensor:
    """d_x [T, H]: the sum of every token's rows of d_rows [T*top_k, H]."""
    ld = _pitched(d_rows, "d_rows")
    T, H = slot_row.shape[0], d_rows.shape[1]
    k = _slots(slot_row, T, d_rows.device)
    if d_rows.shape[0] != T * k:
        raise ValueError(f"d_rows has {d_rows.shape[0]} rows, slot_row {T * k} slots")
    d_x = _out(out, T, H, d_rows.dtype, d_rows.device, stream)
    _check("moe_dispatch_backward", lib().moe_dispatch_backward(
        d_rows.data_ptr(), _DTYPE[d_rows.dtype], T, H, ld, slot_row.data_ptr(), k, d_x.data_ptr(),
        _stream(stream)))
    return d_x


def moe_combine(rows: torch.Tensor, slot_row: torch.Tensor, weights: Optional[torch.Tensor] = None,
                out=None, stream=None) -> torch.Tensor:
    """out [T, H] = sum over a token's slots of weights * rows[slot_row]
    (weights float32 [T, top_k]; None: all 1); dropped slots are left out."""
    ld = _pitched(rows, "rows")
    T, H = slot_row.shape[0], rows.shape[1]
    k = _slots(slot_row, T, rows.device)
    if rows.shape[0] != T * k:
        raise ValueError(f"rows has {rows.shape[0]} rows, slot_row {T * k} slots")
    if weights is not None:
        _exact(weights, "weights", (T, k), torch.float32, rows.device)
    C = _out(out, T, H, rows.dtype, rows.device, stream)
    _check("moe_combine", lib().moe_combine(rows.data_ptr(), _DTYPE[rows.dtype], T, H, ld,
                                            slot_row.data_ptr(), _ptr(weights), k, C.data_ptr(),
                                            _stream(stream)))
    return C


def moe_combine_backward(d_out: torch.Tensor, rows: torch.Tensor, slot_row: torch.Tensor,
                         weights: torch.Tensor, need_d_weights: bool = True, out=None, stream=None):
    """Gradients of moe_combine: (d_rows [T*top_k, H], d_weights float32 [T,
    top_k], or None without ``need_d_weights``, when rows is not read).  ``out``
    may be rows itself."""
    ldd, ld = _pitched(d_out, "d_out"), _pitched(rows, "rows")
    T, H = d_out.shape
    k = _slots(slot_row, T, d_out.device)
    if tuple(rows.shape) != (T * k, H) or rows.dtype != d_out.dtype or rows.device != d_out.device:
        raise ValueError(f"rows must be a {d_out.dtype} tensor of shape ({T * k}, {H}) on {d_out.device}")
    _exact(weights, "weights", (T, k), torch.float32, d_out.device)
    d_rows = _out(out, T * k, H, d_out.dtype, d_out.device, stream)
    dw = _new((T, k), torch.float32, d_out.device, stream) if need_d_weights else None
    _check("moe_combine_backward", lib().moe_combine_backward(
        d_out.data_ptr(), _DTYPE[d_out.dtype], T, H, ldd, rows.data_ptr(), ld,
        slot_row.data_ptr(), weights.data_ptr(), k, d_rows.data_ptr(), _ptr(dw), _stream(stream)))
    return d_rows, dw


# --------------------------------------------------------------------------- 8-bit checkpoints

def quantize_fp8_checkpoint(x: torch.Tensor, stream=None):
    """8-bit checkpoint of x [rows, K] (any row pitch) -> (codes u8 [rows, K]
    E4M3, scales float32 [rows, ceil(K/128)], powers of two)."""
    ld = _pitched(x, "x")
    rows, K = x.shape
    codes = _new((rows, K), torch.uint8, x.device, stream)
    scales = _new((rows, -(-K // 128)), torch.float32, x.device, stream)
    _check("quantize_fp8_checkpoint", lib().quantize_fp8_checkpoint(
        x.data_ptr(), _DTYPE[x.dtype], rows, K, ld, codes.data_ptr(), scales.data_ptr(),
        _stream(stream)))
    return codes, scales


def swiglu_fp8(gate_up: torch.Tensor, out=None, stream=None):
    """h = silu(gate) * up of gate_up = [gate | up] [rows, 2I], and gate_up's
    8-bit checkpoint from the same pass -> (h [rows, I], codes u8 [rows, 2I],
    scales float32 [rows, 2 ceil(I/128)])."""
    ld = _pitched(gate_up, "gate_up")
    rows, two = gate_up.shape
    if two % 2:
        raise ValueError("gate_up must have an even number of columns")
    inner, dev = two // 2, gate_up.device
    h = _out(out, rows, inner, gate_up.dtype, dev, stream)
    codes = _new((rows, two), torch.uint8, dev, stream)
    scales = _new((rows, 2 * -(-inner // 128)), torch.float32, dev, stream)
    _check("swiglu_fp8", lib().swiglu_fp8(
        gate_up.data_ptr(), _DTYPE[gate_up.dtype], rows, inner, ld, h.data_ptr(),
        codes.data_ptr(), scales.data_ptr(), _stream(stream)))
    return h, codes, scales


def swiglu_fp8_backward(d_h: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, out=None,
                        stream=None) -> torch.Tensor:
    """d_gate_up [rows, 2I] from d_h [rows, I] and swiglu_fp8's checkpoint."""
    ld = _pitched(d_h, "d_h")
    rows, inner = d_h.shape
    _exact(codes, "codes", (rows, 2 * inner), torch.uint8, d_h.device)
    _exact(scales, "scales", (rows, 2 * -(-inner // 128)), torch.float32, d_h.device)
    d = _out(out, rows, 2 * inner, d_h.dtype, d_h.device, stream)
    _check("swiglu_fp8_backward", lib().swiglu_fp8_backward(
        d_h.data_ptr(), _DTYPE[d_h.dtype], rows, inner, ld, codes.data_ptr(),
        scales.data_ptr(), d.data_ptr(), _stream(stream)))
    return d


def wgrad_workspace(R: int, N: int, K: int, E: int, device, stream=None) -> torch.Tensor:
    return _empty(max(int(lib().q4_workspace_size_wgrad(R, N, K, E)), 256), device, stream)


def grouped_wgrad_fp8(d_y: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                      expert_offsets: torch.Tensor, row_token: Optional[torch.Tensor] = None,
                      out_dtype=torch.float32, out=None, accumulate: bool = False,
                      ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """dW [E, N, K] = per expert, d_y[rows]^T . x[row_token[rows]] with x the
    checkpoint (codes u8 [T, K], scales [T, ceil(K/128)]).  d_y bf16 [R, N] (any
    row pitch that is a multiple of 8); row_token int32 [R], or None when the
    checkpoint is in row order.  out_dtype float32 or bfloat16; ``accumulate``
    (float32 ``out`` only) adds to ``out``.  ``ws`` from
    ``wgrad_workspace(R, N, K, E, device)``."""
    if d_y.dtype != torch.bfloat16:
        raise ValueError("d_y must be bfloat16")
    ldy = _pitched(d_y, "d_y")
    R, N = d_y.shape
    dev = d_y.device
    _cuda2d(codes, "codes")
    T, K = codes.shape
    _exact(codes, "codes", (T, K), torch.uint8, dev)
    _exact(scales, "scales", (T, -(-K // 128)), torch.float32, dev)
    E = expert_offsets.numel() - 1
    if E < 0:
        raise ValueError("expert_offsets must hold E + 1 entries")
    _exact(expert_offsets, "expert_offsets", (E + 1,), torch.int32, dev)
    if row_token is not None:
        _exact(row_token, "row_token", (R,), torch.int32, dev)
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    if out is None:
        out = _new((E, N, K), out_dtype, dev, stream)
    else:
        _given(_exact(out, "out", (E, N, K), out.dtype, dev), stream)
    if out.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("the gradient is float32 or bfloat16")
    if ws is None:
        ws = wgrad_workspace(R, N, K, E, dev, stream)
    else:
        _given(ws, stream)
    _check("grouped_wgrad_fp8", lib().grouped_wgrad_fp8(
        d_y.data_ptr(), R, N, ldy, codes.data_ptr(), scales.data_ptr(), T, K, _ptr(row_token),
        expert_offsets.data_ptr(), E, out.data_ptr(), _DTYPE[out.dtype], int(accumulate),
        ws.data_ptr(), ws.numel(), _stream(stream)))
    return out


def sync_status(stream=None) -> int:
    """Synchronize and return (and clear) the first error latched by a kernel."""
    return int(lib().q4_sync_status(_stream(stream)))


def set_wait_timeout_ms(ms: int) -> int:
    return int(lib().q4_set_wait_timeout_ms(ms))


def read_probe(src: torch.Tensor, sink: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Measurement aid: one bare streaming read of ``src`` (q4_read_probe).
    Returns the sink (int32 words, contents meaningless)."""
    if not src.is_cuda or not src.is_contiguous():
        raise ValueError("src must be a contiguous CUDA tensor")
    if sink is None:
        sink = _new(int(lib().q4_read_probe_sink_words()), torch.int32, src.device, stream)
        with torch.cuda.stream(stream):
            sink.zero_()
    _check("q4_read_probe", lib().q4_read_probe(src.data_ptr(), src.numel() * src.element_size(),
                                                sink.data_ptr(), _stream(stream)))
    return sink
