"""Thin Python binding of libdg.so (argument marshalling only).

Every step of the computation runs in the library's CUDA kernels; this module only
passes device pointers, sizes and the current CUDA stream through the C ABI
declared in include/dg.h, and allocates outputs with torch when the caller did not
pass them.  There is no fallback: if libdg.so is missing or the device is not
sm_100a, the calls raise.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdg.so")

DG_OK = 0
STATUS_NAMES = {0: "DG_OK", 1: "DG_ERR_INVALID_ARG", 2: "DG_ERR_SHAPE", 3: "DG_ERR_ALIGNMENT",
                4: "DG_ERR_UNSUPPORTED_DEVICE", 5: "DG_ERR_CUDA", 6: "DG_ERR_TIMEOUT",
                7: "DG_ERR_GROUP_OFFSETS"}
KERNELS = {"auto": 0, "tile": 1, "skinny": 2, "pair": 3, "fused": 4}

# every symbol include/dg.h declares
EXPORTS = ("dg_quantize_blockwise", "dg_quantize_blockwise_masked", "dg_fp8_gemm_blockscaled",
           "dg_fp8_gemm_blockscaled_bf16a",
           "dg_fp8_gemm_blockscaled_bf16a_select",
           "dg_fp8_grouped_gemm_contiguous", "dg_fp8_grouped_gemm_masked", "dg_quantize_1x128",
           "dg_fp8_gemm_1x128", "dg_fp8_gemm_1x128_select",
           "dg_fp8_gemm_blockscaled_select", "dg_status_string", "dg_get_last_device_status",
           "dg_version", "dg_test_set_kernel_control",
           "dg_moe_sort", "dg_moe_sort_masked", "dg_moe_sort_workspace", "dg_moe_dispatch_quantize", "dg_moe_dispatch_quantize_masked",
           "dg_moe_combine", "dg_moe_combine_backward", "dg_swiglu_quantize", "dg_swiglu_quantize_masked",
           "dg_swiglu_quantize_backward", "dg_fp8_dgrad_blockscaled", "dg_fp8_wgrad_blockscaled",
           "dg_fp8_grouped_dgrad_contiguous", "dg_fp8_grouped_wgrad_contiguous")


class DGError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)}")


_lib = None


def lib() -> ctypes.CDLL:
    """Load libdg.so once; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing; build it with "
                           "`python -m fp8_block_scaled_scales_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    L.dg_quantize_blockwise.argtypes = [vp, i64, i64, vp, vp, vp]
    L.dg_quantize_blockwise_masked.argtypes = [vp, i32, i64, i64, vp, vp, vp, vp]
    L.dg_fp8_gemm_blockscaled.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, vp]
    L.dg_fp8_gemm_blockscaled_select.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i32, vp]
    L.dg_fp8_gemm_blockscaled_bf16a.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, vp]
    L.dg_fp8_gemm_blockscaled_bf16a_select.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i32, vp]
    L.dg_fp8_grouped_gemm_contiguous.argtypes = [vp, vp, vp, vp, vp, vp, i64, i32, i64, i64, vp]
    L.dg_fp8_grouped_gemm_masked.argtypes = [vp, vp, vp, vp, vp, vp, i32, i64, i64, i64, vp]
    L.dg_quantize_1x128.argtypes = [vp, i64, i64, vp, vp, vp]
    L.dg_fp8_gemm_1x128.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, vp]
    L.dg_fp8_gemm_1x128_select.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i32, vp]
    for f in ("dg_quantize_blockwise", "dg_quantize_blockwise_masked", "dg_fp8_gemm_blockscaled",
              "dg_fp8_gemm_blockscaled_select",
              "dg_fp8_gemm_blockscaled_bf16a", "dg_fp8_gemm_blockscaled_bf16a_select",
              "dg_fp8_grouped_gemm_contiguous", "dg_fp8_grouped_gemm_masked", "dg_get_last_device_status",
              "dg_quantize_1x128", "dg_fp8_gemm_1x128", "dg_fp8_gemm_1x128_select"):
        getattr(L, f).restype = ctypes.c_int
    L.dg_moe_sort.argtypes = [vp, i32, i64, i32, i32, vp, vp, vp, i64, vp, i64, vp]
    L.dg_moe_sort_masked.argtypes = [vp, i32, i64, i32, i32, vp, vp, vp, i64, vp, i64, vp]
    L.dg_moe_sort_workspace.argtypes = [i64, i32, i32]
    L.dg_moe_dispatch_quantize.argtypes = [vp, vp, vp, vp, i64, i32, i64, i64, i32, vp, vp, vp]
    L.dg_moe_dispatch_quantize_masked.argtypes = [vp, vp, vp, i64, i32, i64, i32, i64, vp, vp, vp]
    L.dg_moe_combine.argtypes = [vp, vp, vp, i64, i32, i64, i64, vp, vp]
    L.dg_moe_combine_backward.argtypes = [vp, vp, vp, i64, i32, i64, i64, vp, vp]
    L.dg_swiglu_quantize.argtypes = [vp, vp, i32, i64, i64, vp, vp, vp, vp, vp]
    L.dg_swiglu_quantize_masked.argtypes = [vp, vp, i32, i64, i64, vp, vp, vp]
    L.dg_swiglu_quantize_backward.argtypes = [vp, vp, vp, vp, i32, i64, i64, vp, vp, vp]
    L.dg_fp8_dgrad_blockscaled.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, vp]
    L.dg_fp8_wgrad_blockscaled.argtypes = [vp, vp, vp, vp, vp, i32, i32, i64, i64, i64, vp]
    L.dg_fp8_grouped_dgrad_contiguous.argtypes = [vp, vp, vp, vp, vp, vp, i64, i32, i64, i64, vp]
    L.dg_fp8_grouped_wgrad_contiguous.argtypes = [vp, vp, vp, vp, vp, i32, i32, vp, i64, i32, i64, i64, vp]
    for f in EXPORTS:
        if f.startswith(("dg_moe_", "dg_swiglu_")) or "grad" in f:
            getattr(L, f).restype = ctypes.c_int
    L.dg_moe_sort_workspace.restype = i64
    L.dg_get_last_device_status.argtypes = [vp]
    L.dg_status_string.restype = ctypes.c_char_p
    L.dg_status_string.argtypes = [ctypes.c_int]
    L.dg_version.restype = ctypes.c_int
    L.dg_version.argtypes = []
    L.dg_test_set_kernel_control.restype = None
    L.dg_test_set_kernel_control.argtypes = [ctypes.c_uint64, ctypes.c_int]
    _lib = L
    return L


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _p(t: torch.Tensor | None) -> ctypes.c_void_p:
    if t is None:
        return ctypes.c_void_p(0)
    if not t.is_cuda:
        raise ValueError("tensors must be CUDA device tensors")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous (row-major)")
    return ctypes.c_void_p(t.data_ptr())


def _check(status: int, what: str):
    if status != DG_OK:
        raise DGError(status, what)


def _u8(t: torch.Tensor) -> torch.Tensor:
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def quantize_blockwise(x: torch.Tensor, q: torch.Tensor | None = None, s: torch.Tensor | None = None,
                       stream=None):
    """BF16 [R][C] -> (E4M3 codes uint8 [R][C], FP32 scales [ceil(R/128)][ceil(C/128)])."""
    if x.dtype != torch.bfloat16 or x.dim() != 2:
        raise ValueError("x must be a 2-D bfloat16 tensor")
    R, C = x.shape
    if q is None:
        q = torch.empty((R, C), dtype=torch.uint8, device=x.device)
    if s is None:
        s = torch.empty(((R + 127) // 128, (C + 127) // 128), dtype=torch.float32, device=x.device)
    _check(lib().dg_quantize_blockwise(_p(x), R, C, _p(_u8(q)), _p(s), _stream(stream)),
           "dg_quantize_blockwise")
    return q, s


def quantize_blockwise_masked(x, masked_m, q=None, s=None, stream=None):
    """Block quantization of masked-MoE activations x [G][M_max][K] (bf16): the first
    masked_m[g] rows of slab g (int32 [G] on the device) as quantize_blockwise would
    quantize them alone; rows past the count and the blocks past the last token are
    neither read nor written."""
    G, M_max, K = x.shape
    if q is None:
        q = torch.zeros((G, M_max, K), dtype=torch.uint8, device=x.device)
    if s is None:
        s = torch.zeros((G, (M_max + 127) // 128, (K + 127) // 128), dtype=torch.float32, device=x.device)
    _check(lib().dg_quantize_blockwise_masked(_p(x), G, M_max, K, _p(masked_m), _p(_u8(q)), _p(s), _stream(stream)),
           "dg_quantize_blockwise_masked")
    return q, s


def gemm_blockscaled(A, sA, B, sB, C=None, kernel: str = "auto", stream=None):
    """C[M][N] (bf16) = block-scaled A[M][K] . B[N][K]^T."""
    A, B = _u8(A), _u8(B)
    M, K = A.shape
    N = B.shape[0]
    if C is None:
        C = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    _check(lib().dg_fp8_gemm_blockscaled_select(_p(A), _p(sA), _p(B), _p(sB), _p(C), M, N, K,
                                                KERNELS[kernel], _stream(stream)),
           "dg_fp8_gemm_blockscaled")
    return C


def gemm_blockscaled_bf16a(A, B, sB, C=None, QA=None, sA=None, kernel: str = "auto", stream=None):
    """C[M][N] (bf16) = quantize(A)[M][K] . B[N][K]^T from BF16 activations A.

    Returns (C, QA, sA): A's E4M3 codes and 128x128 block scales are outputs too.
    kernel="fused" (M <= 16) quantizes A inside the skinny GEMM, in one launch."""
    M, K = A.shape
    B = _u8(B)
    N = B.shape[0]
    dev = A.device
    if C is None:
        C = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    if QA is None:
        QA = torch.empty((M, K), dtype=torch.uint8, device=dev)
    if sA is None:
        sA = torch.empty(((M + 127) // 128, (K + 127) // 128), dtype=torch.float32, device=dev)
    _check(lib().dg_fp8_gemm_blockscaled_bf16a_select(_p(A), _p(B), _p(sB), _p(C), _p(_u8(QA)), _p(sA), M, N, K,
                                                      KERNELS[kernel], _stream(stream)),
           "dg_fp8_gemm_blockscaled_bf16a")
    return C, QA, sA


def grouped_gemm_contiguous(A, sA, B, sB, offsets, C=None, stream=None):
    """Grouped-contiguous MoE GEMM: A [M_cap][K], B [G][N][K], offsets int32 [G+1] (device)."""
    A, B = _u8(A), _u8(B)
    Mcap, K = A.shape
    G, N, _ = B.shape
    if C is None:
        C = torch.empty((Mcap, N), dtype=torch.bfloat16, device=A.device)
    _check(lib().dg_fp8_grouped_gemm_contiguous(_p(A), _p(sA), _p(B), _p(sB), _p(C), _p(offsets), Mcap, G,
                                                N, K, _stream(stream)),
           "dg_fp8_grouped_gemm_contiguous")
    return C


def quantize_1x128(x: torch.Tensor, q: torch.Tensor | None = None, s_t: torch.Tensor | None = None,
                   stream=None):
    """BF16 [R][C] -> (E4M3 codes [R][C], FP32 scales [ceil(C/128)][R]), one per row and group."""
    R, C = x.shape
    if q is None:
        q = torch.empty((R, C), dtype=torch.uint8, device=x.device)
    if s_t is None:
        s_t = torch.empty(((C + 127) // 128, R), dtype=torch.float32, device=x.device)
    _check(lib().dg_quantize_1x128(_p(x), R, C, _p(_u8(q)), _p(s_t), _stream(stream)), "dg_quantize_1x128")
    return q, s_t


def gemm_1x128(A, sA_t, B, sB, C=None, kernel: str = "auto", stream=None):
    """C[M][N] (bf16) from A with per-token scales sA_t [ceil(K/128)][M] and 128x128 B scales."""
    A, B = _u8(A), _u8(B)
    M, K = A.shape
    N = B.shape[0]
    if C is None:
        C = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    _check(lib().dg_fp8_gemm_1x128_select(_p(A), _p(sA_t), _p(B), _p(sB), _p(C), M, N, K, KERNELS[kernel],
                                          _stream(stream)),
           "dg_fp8_gemm_1x128")
    return C


def grouped_gemm_masked(A, sA, B, sB, masked_m, C=None, stream=None):
    """Masked MoE GEMM: A [G][M_max][K], B [G][N][K], masked_m int32 [G] (device).

    Rows at or past masked_m[g] of C are not written (a new C is zero-filled)."""
    A, B = _u8(A), _u8(B)
    G, Mmax, K = A.shape
    N = B.shape[1]
    if C is None:
        C = torch.zeros((G, Mmax, N), dtype=torch.bfloat16, device=A.device)
    _check(lib().dg_fp8_grouped_gemm_masked(_p(A), _p(sA), _p(B), _p(sB), _p(C), _p(masked_m), G, Mmax, N, K,
                                            _stream(stream)),
           "dg_fp8_grouped_gemm_masked")
    return C


# ------------------------------------------------------------------- expert layer
_U8, _F32, _BF16, _I32, _I64 = torch.uint8, torch.float32, torch.bfloat16, torch.int32, torch.int64


def _arg(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple, dev: int) -> int:
    """Address of a tensor that has to have this type, shape and device, row-major; codes
    may be uint8 or float8_e4m3fn."""
    if t.dtype is not dtype and not (dtype is _U8 and t.dtype is torch.float8_e4m3fn):
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, the current device and that of the other tensors")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (row-major)")
    return t.data_ptr()


def _out(t, name: str, dtype: torch.dtype, shape: tuple, dev: int):
    """The caller's output, checked, or a new one (not filled): (tensor, address)."""
    if t is None:
        # with its strides given, an allocation takes 1.6 us of host time instead of 2.5
        n = len(shape)
        strides = (1,) if n == 1 else (shape[1], 1) if n == 2 else (shape[1] * shape[2], shape[2], 1)
        t = torch.empty_strided(shape, strides, dtype=dtype, device=_devices(dev))
        return t, t.data_ptr()
    return t, _arg(t, name, dtype, shape, dev)


@functools.lru_cache(maxsize=None)
def _devices(dev: int) -> torch.device:
    return torch.device("cuda", dev)


def _dims(t: torch.Tensor, name: str, n: int):
    """The device of a call's first tensor, which has to be the current one, and its shape."""
    if t.dim() != n:
        raise ValueError(f"{name} must have {n} dimensions, not {t.dim()}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA device tensor")
    dev = t.get_device()
    if dev != torch.cuda.current_device():
        raise ValueError(f"{name} is on cuda:{dev}, which is not the current device")
    return (dev, *t.shape)


# the current stream's handle without building a Stream object (1.3 us of host time a call)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _on(stream, dev: int) -> int:
    """The handle of `stream`, or of the current one."""
    if stream is None:
        return _current_stream(dev)
    return stream.cuda_stream


def _blocks(n: int) -> int:
    return (n + 127) // 128


def moe_capacity(T: int, k: int, G: int) -> int:
    """Rows that T x k slots sorted by G experts can take at most in the contiguous layout."""
    S = T * k
    return (S + 127 * min(G, S)) // 128 * 128


def _sort_workspace(T: int, k: int, G: int, dev: int, stream):
    """Scratch for one sort: (tensor kept alive by the caller, address, bytes)."""
    n = lib().dg_moe_sort_workspace(T, k, G)
    if n == 0:
        return None, 0, 0
    w, p = _out(None, "workspace", _I32, (n // 4,), dev)
    if stream is not None:
        w.record_stream(stream)  # freed here, perhaps while that stream still runs the sort
    return w, p, n


def moe_sort(topk_ids, G: int, offsets=None, row_of_slot=None, slot_of_row=None, stream=None):
    """Slots sorted by expert: topk_ids [T][k] (int32 or int64) -> (group_offsets [G+1],
    row_of_slot [T][k], slot_of_row [capacity]), int32.  Ids outside [0, G) are dropped (row
    -1); rows without a slot hold -1.  capacity: moe_capacity(T, k, G), or that of a larger
    slot_of_row that is passed."""
    dev, T, k = _dims(topk_ids, "topk_ids", 2)
    wide = topk_ids.dtype is _I64
    ids = _arg(topk_ids, "topk_ids", _I64 if wide else _I32, topk_ids.shape, dev)
    cap = moe_capacity(T, k, G) if slot_of_row is None else slot_of_row.numel()
    offsets, p_off = _out(offsets, "offsets", _I32, (G + 1,), dev)
    row_of_slot, p_row = _out(row_of_slot, "row_of_slot", _I32, (T, k), dev)
    slot_of_row, p_slot = _out(slot_of_row, "slot_of_row", _I32, (cap,), dev)
    w, pw, nw = _sort_workspace(T, k, G, dev, stream)
    _check(lib().dg_moe_sort(ids, wide, T, k, G, p_off, p_row, p_slot, cap, pw, nw, _on(stream, dev)), "dg_moe_sort")
    return offsets, row_of_slot, slot_of_row


def moe_sort_masked(topk_ids, G: int, M_max: int, masked_m=None, row_of_slot=None, slot_of_row=None, stream=None):
    """Slots sorted into slabs of M_max rows: (masked_m [G], row_of_slot [T][k],
    slot_of_row [G * M_max]), int32.  An expert's slots past M_max are dropped."""
    dev, T, k = _dims(topk_ids, "topk_ids", 2)
    wide = topk_ids.dtype is _I64
    ids = _arg(topk_ids, "topk_ids", _I64 if wide else _I32, topk_ids.shape, dev)
    masked_m, p_m = _out(masked_m, "masked_m", _I32, (G,), dev)
    row_of_slot, p_row = _out(row_of_slot, "row_of_slot", _I32, (T, k), dev)
    slot_of_row, p_slot = _out(slot_of_row, "slot_of_row", _I32, (G * M_max,), dev)
    w, pw, nw = _sort_workspace(T, k, G, dev, stream)
    _check(lib().dg_moe_sort_masked(ids, wide, T, k, G, p_m, p_row, p_slot, M_max, pw, nw, _on(stream, dev)),
           "dg_moe_sort_masked")
    return masked_m, row_of_slot, slot_of_row


def moe_dispatch_quantize(x, slot_of_row, offsets, k: int, weights=None, q=None, s=None, stream=None):
    """x [T][H] (bf16) gathered by slot_of_row [capacity] and quantized per 128x128 block:
    (codes [capacity][H], scales [capacity/128][ceil(H/128)]).  weights [T][k] (fp32) multiply
    the rows: the gradient of moe_combine with respect to y, for x = dout.  Rows at or past
    offsets[-1] are not written."""
    dev, T, H = _dims(x, "x", 2)
    px = _arg(x, "x", _BF16, (T, H), dev)
    cap, G = slot_of_row.numel(), offsets.numel() - 1
    ps = _arg(slot_of_row, "slot_of_row", _I32, (cap,), dev)
    po = _arg(offsets, "offsets", _I32, (G + 1,), dev)
    pw = 0 if weights is None else _arg(weights, "weights", _F32, (T, k), dev)
    q, pq = _out(q, "q", _U8, (cap, H), dev)
    s, pS = _out(s, "s", _F32, (_blocks(cap), _blocks(H)), dev)
    _check(lib().dg_moe_dispatch_quantize(px, pw, ps, po, T, k, H, cap, G, pq, pS, _on(stream, dev)),
           "dg_moe_dispatch_quantize")
    return q, s


def moe_dispatch_quantize_masked(x, slot_of_row, masked_m, k: int, q=None, s=None, stream=None):
    """x [T][H] (bf16) gathered into slabs and quantized: (codes [G][M_max][H], scales
    [G][ceil(M_max/128)][ceil(H/128)]); rows past a count are not written."""
    dev, T, H = _dims(x, "x", 2)
    px = _arg(x, "x", _BF16, (T, H), dev)
    G = masked_m.numel()
    M_max = slot_of_row.numel() // G if G else 0
    ps = _arg(slot_of_row, "slot_of_row", _I32, (G * M_max,), dev)
    pm = _arg(masked_m, "masked_m", _I32, (G,), dev)
    q, pq = _out(q, "q", _U8, (G, M_max, H), dev)
    s, pS = _out(s, "s", _F32, (G, _blocks(M_max), _blocks(H)), dev)
    _check(lib().dg_moe_dispatch_quantize_masked(px, ps, pm, T, k, H, G, M_max, pq, pS, _on(stream, dev)),
           "dg_moe_dispatch_quantize_masked")
    return q, s


def moe_combine(y, row_of_slot, weights=None, out=None, stream=None):
    """out [T][H] (bf16): the sum over j of weights[t][j] * y[row_of_slot[t][j]]; y is [rows][H]
    or [G][M_max][H].  Without weights: the gradient of the gather with respect to x."""
    dev, T, k = _dims(row_of_slot, "row_of_slot", 2)
    H = y.shape[-1]
    py = _arg(y, "y", _BF16, y.shape, dev)
    rows = y.numel() // H if H else 0
    pr = _arg(row_of_slot, "row_of_slot", _I32, (T, k), dev)
    pw = 0 if weights is None else _arg(weights, "weights", _F32, (T, k), dev)
    out, po = _out(out, "out", _BF16, (T, H), dev)
    _check(lib().dg_moe_combine(py, pw, pr, T, k, H, rows, po, _on(stream, dev)), "dg_moe_combine")
    return out


def moe_combine_backward(dout, y, row_of_slot, dweights=None, stream=None):
    """dweights [T][k] (fp32): dout[t] . y[row_of_slot[t][j]], 0 for a dropped slot.  (The
    gradient with respect to y: moe_dispatch_quantize(dout, ..., weights=weights).)"""
    dev, T, H = _dims(dout, "dout", 2)
    k = row_of_slot.shape[-1]
    pd = _arg(dout, "dout", _BF16, (T, H), dev)
    py = _arg(y, "y", _BF16, (*y.shape[:-1], H), dev)
    rows = y.numel() // H if H else 0
    pr = _arg(row_of_slot, "row_of_slot", _I32, (T, k), dev)
    dweights, pw = _out(dweights, "dweights", _F32, (T, k), dev)
    _check(lib().dg_moe_combine_backward(pd, py, pr, T, k, H, rows, pw, _on(stream, dev)), "dg_moe_combine_backward")
    return dweights


def swiglu_quantize(h, offsets=None, checkpoint: bool = False, q=None, s=None, h8=None, sh=None, stream=None):
    """silu(gate) * up of h [M][2F] = [gate | up] (bf16), quantized per 128x128 block: (codes
    [M][F], scales [ceil(M/128)][F/128]).  checkpoint=True also returns h in 8 bits for
    swiglu_quantize_backward: (codes [M][2F], scales [2F/128][M]), those of quantize_1x128.
    With offsets (int32 [G+1]) rows at or past offsets[-1] are neither read nor written."""
    dev, M, F2 = _dims(h, "h", 2)
    F = F2 // 2
    ph = _arg(h, "h", _BF16, (M, 2 * F), dev)
    G = 0 if offsets is None else offsets.numel() - 1
    po = 0 if offsets is None else _arg(offsets, "offsets", _I32, (G + 1,), dev)
    q, pq = _out(q, "q", _U8, (M, F), dev)
    s, ps = _out(s, "s", _F32, (_blocks(M), _blocks(F)), dev)
    p8 = psh = 0
    if checkpoint:
        h8, p8 = _out(h8, "h8", _U8, (M, 2 * F), dev)
        sh, psh = _out(sh, "sh", _F32, (2 * F // 128, M), dev)
    elif h8 is not None or sh is not None:
        raise ValueError("h8 and sh are outputs of checkpoint=True")
    _check(lib().dg_swiglu_quantize(ph, po, G, M, F, pq, ps, p8, psh, _on(stream, dev)), "dg_swiglu_quantize")
    return (q, s, h8, sh) if checkpoint else (q, s)


def swiglu_quantize_masked(h, masked_m, q=None, s=None, stream=None):
    """swiglu_quantize for the masked layout: h [G][M_max][2F] -> (codes [G][M_max][F], scales
    [G][ceil(M_max/128)][F/128]); rows past a count are neither read nor written."""
    dev, G, M_max, F2 = _dims(h, "h", 3)
    F = F2 // 2
    ph = _arg(h, "h", _BF16, (G, M_max, 2 * F), dev)
    pm = _arg(masked_m, "masked_m", _I32, (G,), dev)
    q, pq = _out(q, "q", _U8, (G, M_max, F), dev)
    s, ps = _out(s, "s", _F32, (G, _blocks(M_max), _blocks(F)), dev)
    _check(lib().dg_swiglu_quantize_masked(ph, pm, G, M_max, F, pq, ps, _on(stream, dev)),
           "dg_swiglu_quantize_masked")
    return q, s


def swiglu_quantize_backward(h8, sh, da, offsets=None, q=None, s=None, stream=None):
    """Gradient of swiglu with respect to h, from its 8-bit checkpoint (h8 [M][2F], sh
    [2F/128][M]) and da [M][F] (bf16), quantized per 128x128 block: (codes [M][2F], scales
    [ceil(M/128)][2F/128])."""
    dev, M, F = _dims(da, "da", 2)
    p8 = _arg(h8, "h8", _U8, (M, 2 * F), dev)
    psh = _arg(sh, "sh", _F32, (2 * F // 128, M), dev)
    pa = _arg(da, "da", _BF16, (M, F), dev)
    G = 0 if offsets is None else offsets.numel() - 1
    po = 0 if offsets is None else _arg(offsets, "offsets", _I32, (G + 1,), dev)
    q, pq = _out(q, "q", _U8, (M, 2 * F), dev)
    s, ps = _out(s, "s", _F32, (_blocks(M), _blocks(2 * F)), dev)
    _check(lib().dg_swiglu_quantize_backward(p8, psh, pa, po, G, M, F, pq, ps, _on(stream, dev)),
           "dg_swiglu_quantize_backward")
    return q, s


def dgrad_blockscaled(dY, sdY, W, sW, C=None, stream=None):
    """Input gradient C [M][K] (bf16) of a dense layer: codes dY [M][N] times the weights'
    codes W [N][K], both as the forward pass has them."""
    dev, M, N = _dims(dY, "dY", 2)
    K = W.shape[-1]
    pd = _arg(dY, "dY", _U8, (M, N), dev)
    pa = _arg(sdY, "sdY", _F32, (_blocks(M), _blocks(N)), dev)
    pw = _arg(W, "W", _U8, (N, K), dev)
    pb = _arg(sW, "sW", _F32, (_blocks(N), _blocks(K)), dev)
    C, pc = _out(C, "C", _BF16, (M, K), dev)
    _check(lib().dg_fp8_dgrad_blockscaled(pd, pa, pw, pb, pc, M, N, K, _on(stream, dev)), "dg_fp8_dgrad_blockscaled")
    return C


def grouped_dgrad_contiguous(dY, sdY, W, sW, offsets, C=None, stream=None):
    """Input gradient expert by expert: dY [M_cap][N], W [G][N][K], offsets int32 [G+1] ->
    C [M_cap][K] (bf16); rows at or past offsets[-1] are not written."""
    dev, M, N = _dims(dY, "dY", 2)
    G, K = offsets.numel() - 1, W.shape[-1]
    pd = _arg(dY, "dY", _U8, (M, N), dev)
    pa = _arg(sdY, "sdY", _F32, (_blocks(M), _blocks(N)), dev)
    pw = _arg(W, "W", _U8, (G, N, K), dev)
    pb = _arg(sW, "sW", _F32, (G, _blocks(N), _blocks(K)), dev)
    po = _arg(offsets, "offsets", _I32, (G + 1,), dev)
    C, pc = _out(C, "C", _BF16, (M, K), dev)
    _check(lib().dg_fp8_grouped_dgrad_contiguous(pd, pa, pw, pb, pc, po, M, G, N, K, _on(stream, dev)),
           "dg_fp8_grouped_dgrad_contiguous")
    return C


def _wgrad_out(C, dtype, accumulate: bool, shape: tuple, dev: int):
    if C is not None:
        dtype = C.dtype if dtype is None else dtype
    elif accumulate:
        raise ValueError("accumulate needs the gradient C that is added to")
    dtype = _F32 if dtype is None else dtype
    if dtype not in (_F32, _BF16):
        raise ValueError("a weight gradient is float32 or bfloat16")
    C, pc = _out(C, "C", dtype, shape, dev)
    return C, pc, dtype is _F32


def wgrad_blockscaled(dY, sdY, X, sX, C=None, accumulate: bool = False, dtype=None, stream=None):
    """Weight gradient C [N][K] (float32, or dtype=torch.bfloat16) of a dense layer: codes dY
    [M][N] and the forward input's codes X [M][K].  accumulate=True adds to C (float32)."""
    dev, M, N = _dims(dY, "dY", 2)
    K = X.shape[-1]
    pd = _arg(dY, "dY", _U8, (M, N), dev)
    pa = _arg(sdY, "sdY", _F32, (_blocks(M), _blocks(N)), dev)
    px = _arg(X, "X", _U8, (M, K), dev)
    pb = _arg(sX, "sX", _F32, (_blocks(M), _blocks(K)), dev)
    C, pc, f32 = _wgrad_out(C, dtype, accumulate, (N, K), dev)
    _check(lib().dg_fp8_wgrad_blockscaled(pd, pa, px, pb, pc, f32, accumulate, M, N, K, _on(stream, dev)),
           "dg_fp8_wgrad_blockscaled")
    return C


def grouped_wgrad_contiguous(dY, sdY, X, sX, offsets, C=None, accumulate: bool = False, dtype=None, stream=None):
    """Weight gradients C [G][N][K] expert by expert, from rows [offsets[g], offsets[g+1]) of dY
    [M_cap][N] and X [M_cap][K]; an expert without rows gets zeros (accumulate: keeps its C)."""
    dev, M, N = _dims(dY, "dY", 2)
    G, K = offsets.numel() - 1, X.shape[-1]
    pd = _arg(dY, "dY", _U8, (M, N), dev)
    pa = _arg(sdY, "sdY", _F32, (_blocks(M), _blocks(N)), dev)
    px = _arg(X, "X", _U8, (M, K), dev)
    pb = _arg(sX, "sX", _F32, (_blocks(M), _blocks(K)), dev)
    po = _arg(offsets, "offsets", _I32, (G + 1,), dev)
    C, pc, f32 = _wgrad_out(C, dtype, accumulate, (G, N, K), dev)
    _check(lib().dg_fp8_grouped_wgrad_contiguous(pd, pa, px, pb, pc, f32, accumulate, po, M, G, N, K,
                                                 _on(stream, dev)),
           "dg_fp8_grouped_wgrad_contiguous")
    return C


def last_device_status(stream=None) -> int:
    """Synchronise and return (and clear) the library's device status word."""
    return lib().dg_get_last_device_status(_stream(stream))


def set_kernel_control(timeout_ns: int = 0, debug_flags: int = 0):
    lib().dg_test_set_kernel_control(timeout_ns, debug_flags)


def version() -> int:
    return lib().dg_version()
