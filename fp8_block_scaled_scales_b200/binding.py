"""Thin Python binding of libdg.so (argument marshalling only).

Every step of the computation runs in the library's CUDA kernels; this module only
passes device pointers, sizes and the current CUDA stream through the C ABI
declared in include/dg.h, and allocates outputs with torch when the caller did not
pass them.  There is no fallback: if libdg.so is missing or the device is not
sm_100a, the calls raise.
"""
from __future__ import annotations

import ctypes
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
           "dg_moe_sort", "dg_moe_sort_masked", "dg_moe_sort_workspace", "dg_moe_dispatch_quantize", "dg_moe_dispatch_workspace", "dg_moe_dispatch_quantize_masked",
           "dg_moe_combine", "dg_moe_combine_backward", "dg_swiglu_quantize", "dg_swiglu_quantize_masked",
           "dg_swiglu_quantize_backward", "dg_fp8_dgrad_blockscaled", "dg_fp8_dgrad_workspace", "dg_fp8_wgrad_blockscaled",
           "dg_fp8_wgrad_workspace",
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
    L.dg_moe_dispatch_quantize.argtypes = [vp, vp, vp, vp, i64, i32, i64, i64, i32, vp, vp, vp, i64, vp]
    L.dg_moe_dispatch_workspace.argtypes = [i64, i32, i64, i64]
    L.dg_moe_dispatch_quantize_masked.argtypes = [vp, vp, vp, i64, i32, i64, i32, i64, vp, vp, vp]
    L.dg_moe_combine.argtypes = [vp, vp, vp, i64, i32, i64, i64, vp, vp]
    L.dg_moe_combine_backward.argtypes = [vp, vp, vp, i64, i32, i64, i64, vp, vp]
    L.dg_swiglu_quantize.argtypes = [vp, vp, i32, i64, i64, vp, vp, vp, vp, vp]
    L.dg_swiglu_quantize_masked.argtypes = [vp, vp, i32, i64, i64, vp, vp, vp]
    L.dg_swiglu_quantize_backward.argtypes = [vp, vp, vp, vp, i32, i64, i64, vp, vp, vp]
    L.dg_fp8_dgrad_blockscaled.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, vp, i64, vp]
    L.dg_fp8_wgrad_blockscaled.argtypes = [vp, vp, vp, vp, vp, i32, i32, i64, i64, i64, vp, i64, vp]
    L.dg_fp8_dgrad_workspace.argtypes = L.dg_fp8_wgrad_workspace.argtypes = [i64, i64, i64]
    L.dg_fp8_grouped_dgrad_contiguous.argtypes = [vp, vp, vp, vp, vp, vp, i64, i32, i64, i64, vp]
    L.dg_fp8_grouped_wgrad_contiguous.argtypes = [vp, vp, vp, vp, vp, i32, i32, vp, i64, i32, i64, i64, vp]
    for f in EXPORTS:
        if f.startswith(("dg_moe_", "dg_swiglu_")) or "grad" in f:
            getattr(L, f).restype = ctypes.c_int
    for f in (L.dg_moe_sort_workspace, L.dg_moe_dispatch_workspace, L.dg_fp8_dgrad_workspace, L.dg_fp8_wgrad_workspace):
        f.restype = i64
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


def _new(shape, dtype, device, stream, filled: bool = False) -> torch.Tensor:
    """An output, allocated (and zero-filled) on the stream of the call: on the current one, the memory
    could still be in use there, and the fill would not come before the call's kernel."""
    make = torch.zeros if filled else torch.empty
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=device)
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=device)


def quantize_blockwise(x: torch.Tensor, q: torch.Tensor | None = None, s: torch.Tensor | None = None,
                       stream=None):
    """BF16 [R][C] -> (E4M3 codes uint8 [R][C], FP32 scales [ceil(R/128)][ceil(C/128)])."""
    if x.dtype != torch.bfloat16 or x.dim() != 2:
        raise ValueError("x must be a 2-D bfloat16 tensor")
    R, C = x.shape
    if q is None:
        q = _new((R, C), torch.uint8, x.device, stream)
    if s is None:
        s = _new(((R + 127) // 128, (C + 127) // 128), torch.float32, x.device, stream)
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
        q = _new((G, M_max, K), torch.uint8, x.device, stream, filled=True)
    if s is None:
        s = _new((G, (M_max + 127) // 128, (K + 127) // 128), torch.float32, x.device, stream, filled=True)
    _check(lib().dg_quantize_blockwise_masked(_p(x), G, M_max, K, _p(masked_m), _p(_u8(q)), _p(s), _stream(stream)),
           "dg_quantize_blockwise_masked")
    return q, s


def gemm_blockscaled(A, sA, B, sB, C=None, kernel: str = "auto", stream=None):
    """C[M][N] (bf16) = block-scaled A[M][K] . B[N][K]^T."""
    A, B = _u8(A), _u8(B)
    M, K = A.shape
    N = B.shape[0]
    if C is None:
        C = _new((M, N), torch.bfloat16, A.device, stream)
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
        C = _new((M, N), torch.bfloat16, dev, stream)
    if QA is None:
        QA = _new((M, K), torch.uint8, dev, stream)
    if sA is None:
        sA = _new(((M + 127) // 128, (K + 127) // 128), torch.float32, dev, stream)
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
        C = _new((Mcap, N), torch.bfloat16, A.device, stream)
    _check(lib().dg_fp8_grouped_gemm_contiguous(_p(A), _p(sA), _p(B), _p(sB), _p(C), _p(offsets), Mcap, G,
                                                N, K, _stream(stream)),
           "dg_fp8_grouped_gemm_contiguous")
    return C


def quantize_1x128(x: torch.Tensor, q: torch.Tensor | None = None, s_t: torch.Tensor | None = None,
                   stream=None):
    """BF16 [R][C] -> (E4M3 codes [R][C], FP32 scales [ceil(C/128)][R]), one per row and group."""
    R, C = x.shape
    if q is None:
        q = _new((R, C), torch.uint8, x.device, stream)
    if s_t is None:
        s_t = _new(((C + 127) // 128, R), torch.float32, x.device, stream)
    _check(lib().dg_quantize_1x128(_p(x), R, C, _p(_u8(q)), _p(s_t), _stream(stream)), "dg_quantize_1x128")
    return q, s_t


def gemm_1x128(A, sA_t, B, sB, C=None, kernel: str = "auto", stream=None):
    """C[M][N] (bf16) from A with per-token scales sA_t [ceil(K/128)][M] and 128x128 B scales."""
    A, B = _u8(A), _u8(B)
    M, K = A.shape
    N = B.shape[0]
    if C is None:
        C = _new((M, N), torch.bfloat16, A.device, stream)
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
        C = _new((G, Mmax, N), torch.bfloat16, A.device, stream, filled=True)
    _check(lib().dg_fp8_grouped_gemm_masked(_p(A), _p(sA), _p(B), _p(sB), _p(C), _p(masked_m), G, Mmax, N, K,
                                            _stream(stream)),
           "dg_fp8_grouped_gemm_masked")
    return C


# ------------------------------------------------------------------- expert layer
# These calls check their tensors, allocate what the caller did not pass and call the C ABI in
# native code (csrc/torch_binding.cpp): a chain of short kernels should not wait for Python.
# Tensors of the wrong type, shape, device or layout raise ValueError, what the library
# refuses DGError.  New outputs are not filled.  With stream= a call runs on that stream, and
# what it allocates, outputs and workspaces, is allocated there too, as under
# torch.cuda.stream(stream): the caller orders its other streams around it.
_ext = None


def _native():
    """Load _dgtorch.so once; raises if it has not been built."""
    global _ext
    if _ext is None:
        lib()
        try:
            from . import _dgtorch
        except ImportError as e:
            raise RuntimeError(f"{os.path.join(_HERE, '_dgtorch.so')} is missing or does not load ({e}); build it "
                               "with `python -m fp8_block_scaled_scales_b200.build`") from e
        _dgtorch.set_error(DGError)
        _ext = _dgtorch
    return _ext


def moe_capacity(T: int, k: int, G: int) -> int:
    """Rows that T x k slots sorted by G experts can take at most in the contiguous layout."""
    S = T * k
    return (S + 127 * min(G, S)) // 128 * 128


def moe_sort(topk_ids, G: int, offsets=None, row_of_slot=None, slot_of_row=None, stream=None):
    """Slots sorted by expert: topk_ids [T][k] (int32 or int64) -> (group_offsets [G+1],
    row_of_slot [T][k], slot_of_row [capacity]), int32.  Ids outside [0, G) are dropped (row
    -1); rows without a slot hold -1.  capacity: moe_capacity(T, k, G), or that of a larger
    slot_of_row that is passed."""
    return (_ext or _native()).moe_sort(topk_ids, G, offsets, row_of_slot, slot_of_row, stream)


def moe_sort_masked(topk_ids, G: int, M_max: int, masked_m=None, row_of_slot=None, slot_of_row=None, stream=None):
    """Slots sorted into slabs of M_max rows: (masked_m [G], row_of_slot [T][k],
    slot_of_row [G * M_max]), int32.  An expert's slots past M_max are dropped."""
    return (_ext or _native()).moe_sort_masked(topk_ids, G, M_max, masked_m, row_of_slot, slot_of_row, stream)


def moe_dispatch_quantize(x, slot_of_row, offsets, k: int, weights=None, q=None, s=None, stream=None):
    """x [T][H] (bf16) gathered by slot_of_row [capacity] and quantized per 128x128 block:
    (codes [capacity][H], scales [capacity/128][ceil(H/128)]).  weights [T][k] (fp32) multiply
    the rows: the gradient of moe_combine with respect to y, for x = dout.  Rows at or past
    offsets[-1] are not written."""
    return (_ext or _native()).moe_dispatch_quantize(x, slot_of_row, offsets, k, weights, q, s, stream)


def moe_dispatch_quantize_masked(x, slot_of_row, masked_m, k: int, q=None, s=None, stream=None):
    """x [T][H] (bf16) gathered into slabs and quantized: (codes [G][M_max][H], scales
    [G][ceil(M_max/128)][ceil(H/128)]); rows past a count are not written."""
    return (_ext or _native()).moe_dispatch_quantize_masked(x, slot_of_row, masked_m, k, q, s, stream)


def moe_combine(y, row_of_slot, weights=None, out=None, stream=None):
    """out [T][H] (bf16): the sum over j of weights[t][j] * y[row_of_slot[t][j]]; y is [rows][H]
    or [G][M_max][H].  Without weights: the gradient of the gather with respect to x."""
    return (_ext or _native()).moe_combine(y, row_of_slot, weights, out, stream)


def moe_combine_backward(dout, y, row_of_slot, dweights=None, stream=None):
    """dweights [T][k] (fp32): dout[t] . y[row_of_slot[t][j]], 0 for a dropped slot.  (The
    gradient with respect to y: moe_dispatch_quantize(dout, ..., weights=weights).)"""
    return (_ext or _native()).moe_combine_backward(dout, y, row_of_slot, dweights, stream)


def swiglu_quantize(h, offsets=None, checkpoint: bool = False, q=None, s=None, h8=None, sh=None, stream=None):
    """silu(gate) * up of h [M][2F] = [gate | up] (bf16), quantized per 128x128 block: (codes
    [M][F], scales [ceil(M/128)][F/128]).  checkpoint=True also returns h in 8 bits for
    swiglu_quantize_backward: (codes [M][2F], scales [2F/128][M]), those of quantize_1x128.
    With offsets (int32 [G+1]) rows at or past offsets[-1] are neither read nor written."""
    return (_ext or _native()).swiglu_quantize(h, offsets, checkpoint, q, s, h8, sh, stream)


def swiglu_quantize_masked(h, masked_m, q=None, s=None, stream=None):
    """swiglu_quantize for the masked layout: h [G][M_max][2F] -> (codes [G][M_max][F], scales
    [G][ceil(M_max/128)][F/128]); rows past a count are neither read nor written."""
    return (_ext or _native()).swiglu_quantize_masked(h, masked_m, q, s, stream)


def swiglu_quantize_backward(h8, sh, da, offsets=None, q=None, s=None, stream=None):
    """Gradient of swiglu with respect to h, from its 8-bit checkpoint (h8 [M][2F], sh
    [2F/128][M]) and da [M][F] (bf16), quantized per 128x128 block: (codes [M][2F], scales
    [ceil(M/128)][2F/128])."""
    return (_ext or _native()).swiglu_quantize_backward(h8, sh, da, offsets, q, s, stream)


def dgrad_blockscaled(dY, sdY, W, sW, C=None, stream=None):
    """Input gradient C [M][K] (bf16) of a dense layer: codes dY [M][N] times the weights'
    codes W [N][K], both as the forward pass has them."""
    return (_ext or _native()).dgrad(dY, sdY, W, sW, None, C, stream)


def grouped_dgrad_contiguous(dY, sdY, W, sW, offsets, C=None, stream=None):
    """Input gradient expert by expert: dY [M_cap][N], W [G][N][K], offsets int32 [G+1] ->
    C [M_cap][K] (bf16); rows at or past offsets[-1] are not written."""
    return (_ext or _native()).dgrad(dY, sdY, W, sW, _given(offsets), C, stream)


def _given(offsets):
    if offsets is None:
        raise ValueError("offsets must be a tensor")
    return offsets


_GRAD_DTYPES = {None: None, torch.float32: False, torch.bfloat16: True}


def _grad_dtype(dtype):
    if dtype not in _GRAD_DTYPES:
        raise ValueError("a weight gradient is float32 or bfloat16")
    return _GRAD_DTYPES[dtype]


def wgrad_blockscaled(dY, sdY, X, sX, C=None, accumulate: bool = False, dtype=None, stream=None):
    """Weight gradient C [N][K] (float32, or dtype=torch.bfloat16) of a dense layer: codes dY
    [M][N] and the forward input's codes X [M][K].  accumulate=True adds to C (float32)."""
    return (_ext or _native()).wgrad(dY, sdY, X, sX, None, C, accumulate, _grad_dtype(dtype), stream)


def grouped_wgrad_contiguous(dY, sdY, X, sX, offsets, C=None, accumulate: bool = False, dtype=None, stream=None):
    """Weight gradients C [G][N][K] expert by expert, from rows [offsets[g], offsets[g+1]) of dY
    [M_cap][N] and X [M_cap][K]; an expert without rows gets zeros (accumulate: keeps its C)."""
    return (_ext or _native()).wgrad(dY, sdY, X, sX, _given(offsets), C, accumulate, _grad_dtype(dtype), stream)


def last_device_status(stream=None) -> int:
    """Synchronise and return (and clear) the library's device status word."""
    return lib().dg_get_last_device_status(_stream(stream))


def set_kernel_control(timeout_ns: int = 0, debug_flags: int = 0):
    lib().dg_test_set_kernel_control(timeout_ns, debug_flags)


def version() -> int:
    return lib().dg_version()
