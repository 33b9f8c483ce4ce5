"""Refusals of the expert-layer and gradient calls, decided on the host before any CUDA call."""
import ctypes

import pytest
import torch

from fp8_block_scaled_scales_b200 import binding
from fp8_block_scaled_scales_b200 import build as dgbuild

NULL = ctypes.c_void_p(0)
P = ctypes.c_void_p(0x10000)   # never dereferenced: the refusal comes first
ODD = ctypes.c_void_p(0x10001)
OK, ARG, SHAPE, ALIGN = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    dgbuild.build()
    return binding.lib()


def test_sort_refusals(lib):
    f = lib.dg_moe_sort
    assert f(P, 0, -1, 2, 4, P, P, P, 1024, NULL, 0, NULL) == SHAPE
    assert f(P, 0, 8, 0, 4, P, P, P, 1024, NULL, 0, NULL) == SHAPE              # k == 0
    assert f(P, 0, 8, 2, 0, P, P, P, 1024, NULL, 0, NULL) == SHAPE
    assert f(P, 0, 8, 2, 1025, P, P, P, 1 << 20, NULL, 0, NULL) == SHAPE
    assert f(P, 0, 8, 2, 4, P, P, P, 1000, NULL, 0, NULL) == SHAPE              # capacity % 128
    # 16 slots over 4 experts may take four blocks of 128
    assert f(P, 0, 8, 2, 4, P, P, P, 384, NULL, 0, NULL) == SHAPE
    assert f(P, 0, 1 << 30, 2, 4, P, P, P, 1 << 30, NULL, 0, NULL) == SHAPE     # T * k > 2^30
    assert f(NULL, 0, 8, 2, 4, P, P, P, 512, NULL, 0, NULL) == ARG
    assert f(P, 0, 8, 2, 4, NULL, P, P, 512, NULL, 0, NULL) == ARG
    assert f(P, 0, 8, 2, 4, P, P, NULL, 512, NULL, 0, NULL) == ARG
    assert f(ctypes.c_void_p(0x10004), 1, 8, 2, 4, P, P, P, 512, NULL, 0, NULL) == ALIGN  # int64 ids at 4 bytes
    assert f(P, 0, 8, 2, 4, ODD, P, P, 512, NULL, 0, NULL) == ALIGN
    # more slots than one CTA takes: a workspace of the size that the library names
    need = lib.dg_moe_sort_workspace(8192, 2, 64)
    cap = binding.moe_capacity(8192, 2, 64)
    assert need > 0 and lib.dg_moe_sort_workspace(8, 2, 4) == 0 and lib.dg_moe_sort_workspace(-1, 2, 4) == 0
    assert f(P, 0, 8192, 2, 64, P, P, P, cap, NULL, need, NULL) == ARG
    assert f(P, 0, 8192, 2, 64, P, P, P, cap, P, need - 4, NULL) == ARG
    assert f(P, 0, 8192, 2, 64, P, P, P, cap, ODD, need, NULL) == ALIGN
    m = lib.dg_moe_sort_masked
    assert m(P, 0, 8, 2, 4, P, P, P, -1, NULL, 0, NULL) == SHAPE
    assert m(P, 0, 8, 2, 4, P, P, P, 1 << 30, NULL, 0, NULL) == SHAPE           # G * M_max >= 2^31
    assert m(P, 0, 8, 2, 4, NULL, P, P, 64, NULL, 0, NULL) == ARG
    assert m(P, 0, 8, 2, 4, P, P, ODD, 64, NULL, 0, NULL) == ALIGN


def test_capacity_helper_is_the_least_the_sort_takes(lib):
    for T, k, G in ((1, 8, 64), (1, 1, 1), (100, 2, 3), (8192, 2, 8), (0, 4, 16)):
        cap = binding.moe_capacity(T, k, G)
        if cap:
            assert lib.dg_moe_sort(P, 0, T, k, G, P, P, P, cap - 128, P, 1 << 30, NULL) == SHAPE
        assert lib.dg_moe_sort(P, 0, T, k, G, ODD, P, P, cap, P, 1 << 30, NULL) == ALIGN  # capacity accepted
        # the worst routing fits: every expert one slot, the rest in one, each rounded up
        S = T * k
        used = min(G, S)
        worst = (used - 1) * 128 + -(-(S - used + 1) // 128) * 128 if S else 0
        assert worst <= cap


def test_dispatch_refusals(lib):
    f = lib.dg_moe_dispatch_quantize
    assert f(P, NULL, P, P, 8, 2, 24, 128, 4, P, P, NULL, 0, NULL) == SHAPE     # H % 16
    assert f(P, NULL, P, P, 8, 2, 32, 100, 4, P, P, NULL, 0, NULL) == SHAPE     # capacity % 128
    assert f(P, NULL, P, P, 8, 2, 32, 128, 0, P, P, NULL, 0, NULL) == SHAPE
    assert f(P, NULL, P, P, -1, 2, 32, 128, 4, P, P, NULL, 0, NULL) == SHAPE
    assert f(NULL, NULL, NULL, NULL, 8, 2, 32, 0, 4, NULL, NULL, NULL, 0, NULL) == OK
    assert f(NULL, NULL, NULL, NULL, 8, 2, 0, 128, 4, NULL, NULL, NULL, 0, NULL) == OK
    assert f(P, NULL, NULL, P, 8, 2, 32, 128, 4, P, P, NULL, 0, NULL) == ARG
    assert f(NULL, NULL, P, P, 8, 2, 32, 128, 4, P, P, NULL, 0, NULL) == ARG
    assert f(ODD, NULL, P, P, 8, 2, 32, 128, 4, P, P, NULL, 0, NULL) == ALIGN
    assert f(P, ODD, P, P, 8, 2, 32, 128, 4, P, P, NULL, 0, NULL) == ALIGN
    # many slots a token: a workspace of the size that the library names
    cap = binding.moe_capacity(4096, 8, 64)
    need = lib.dg_moe_dispatch_workspace(4096, 8, 7168, cap)
    assert need >= 4096 * 8 * 4 + cap * 4 + 4096 * 56 * 2 and lib.dg_moe_dispatch_workspace(64, 2, 7168, cap) == 0
    assert lib.dg_moe_dispatch_workspace(-1, 8, 7168, cap) == lib.dg_moe_dispatch_workspace(4096, 8, 7160, cap) == 0
    assert f(P, NULL, P, P, 4096, 8, 7168, cap, 64, P, P, NULL, need, NULL) == ARG
    assert f(P, NULL, P, P, 4096, 8, 7168, cap, 64, P, P, P, need - 1, NULL) == ARG
    assert f(P, NULL, P, P, 4096, 8, 7168, cap, 64, P, P, ODD, need, NULL) == ALIGN
    m = lib.dg_moe_dispatch_quantize_masked
    assert m(P, P, P, 8, 2, 24, 4, 64, P, P, NULL) == SHAPE
    assert m(P, P, P, 8, 2, 32, 1025, 64, P, P, NULL) == SHAPE
    assert m(NULL, NULL, NULL, 8, 2, 32, 4, 0, NULL, NULL, NULL) == OK
    assert m(P, P, NULL, 8, 2, 32, 4, 64, P, P, NULL) == ARG
    assert m(P, P, P, 8, 2, 32, 4, 64, ODD, P, NULL) == ALIGN


def test_combine_refusals(lib):
    f = lib.dg_moe_combine
    assert f(P, P, P, 8, 2, 24, 128, P, NULL) == SHAPE
    assert f(P, P, P, 8, 2, 32, -1, P, NULL) == SHAPE
    assert f(P, P, P, 8, 0, 32, 128, P, NULL) == SHAPE
    assert f(NULL, NULL, NULL, 0, 2, 32, 128, NULL, NULL) == OK
    assert f(NULL, P, P, 8, 2, 32, 128, P, NULL) == ARG
    assert f(P, P, P, 8, 2, 32, 128, NULL, NULL) == ARG
    assert f(P, P, P, 8, 2, 32, 128, ODD, NULL) == ALIGN
    b = lib.dg_moe_combine_backward
    assert b(P, P, P, 8, 2, 24, 128, P, NULL) == SHAPE
    assert b(NULL, NULL, NULL, 0, 2, 32, 128, NULL, NULL) == OK
    assert b(P, P, P, 8, 2, 32, 128, NULL, NULL) == ARG
    assert b(P, ODD, P, 8, 2, 32, 128, P, NULL) == ALIGN


def test_swiglu_refusals(lib):
    f = lib.dg_swiglu_quantize
    assert f(P, NULL, 0, 8, 100, P, P, NULL, NULL, NULL) == SHAPE      # F % 128
    assert f(P, P, 4, 100, 128, P, P, NULL, NULL, NULL) == SHAPE       # grouped: M % 128
    assert f(P, P, 0, 128, 128, P, P, NULL, NULL, NULL) == SHAPE       # grouped: G
    assert f(NULL, NULL, 0, 0, 128, NULL, NULL, NULL, NULL, NULL) == OK
    assert f(P, NULL, 0, 8, 128, P, P, P, NULL, NULL) == ARG           # half a checkpoint
    assert f(P, NULL, 0, 8, 128, NULL, P, NULL, NULL, NULL) == ARG
    assert f(ODD, NULL, 0, 8, 128, P, P, NULL, NULL, NULL) == ALIGN
    m = lib.dg_swiglu_quantize_masked
    assert m(P, P, 0, 8, 128, P, P, NULL) == SHAPE
    assert m(P, NULL, 2, 8, 128, P, P, NULL) == ARG
    assert m(P, ODD, 2, 8, 128, P, P, NULL) == ALIGN
    b = lib.dg_swiglu_quantize_backward
    assert b(P, P, P, NULL, 0, 8, 64, P, P, NULL) == SHAPE
    assert b(P, NULL, P, NULL, 0, 8, 128, P, P, NULL) == ARG
    assert b(P, P, ODD, NULL, 0, 8, 128, P, P, NULL) == ALIGN


def test_gradient_product_refusals(lib):
    d = lib.dg_fp8_dgrad_blockscaled
    assert d(P, P, P, P, P, 8, 0, 128, NULL, 0, NULL) == SHAPE                  # nothing to sum over
    assert d(P, P, P, P, P, 8, 24, 128, NULL, 0, NULL) == SHAPE
    assert d(P, P, P, P, P, 8, 128, 24, NULL, 0, NULL) == SHAPE
    assert d(NULL, NULL, NULL, NULL, NULL, 0, 128, 128, NULL, 0, NULL) == OK
    assert d(P, P, P, P, NULL, 8, 128, 128, NULL, 0, NULL) == ARG
    assert d(P, P, ODD, P, P, 8, 128, 128, NULL, 0, NULL) == ALIGN
    w = lib.dg_fp8_wgrad_blockscaled
    assert w(P, P, P, P, P, 1, 0, 8, 24, 128, NULL, 0, NULL) == SHAPE
    assert w(P, P, P, P, P, 0, 1, 8, 128, 128, NULL, 0, NULL) == ARG            # accumulate in BF16
    assert w(NULL, NULL, NULL, NULL, NULL, 1, 0, 8, 0, 128, NULL, 0, NULL) == OK
    assert w(P, P, P, P, NULL, 1, 0, 8, 128, 128, NULL, 0, NULL) == ARG
    assert w(NULL, NULL, NULL, NULL, NULL, 1, 0, 0, 128, 128, NULL, 0, NULL) == ARG  # M == 0 still writes dW
    assert w(P, P, P, P, ODD, 1, 0, 8, 128, 128, NULL, 0, NULL) == ALIGN
    # few tiles and long sums: a workspace of the size that the library names
    need = lib.dg_fp8_wgrad_workspace(4096, 256, 256)
    assert need >= 2 * 256 * 256 * 4 and lib.dg_fp8_wgrad_workspace(4096, 4096, 4096) == 0
    assert lib.dg_fp8_wgrad_workspace(4096, 250, 256) == lib.dg_fp8_wgrad_workspace(-1, 256, 256) == 0
    assert w(P, P, P, P, P, 1, 0, 4096, 256, 256, NULL, need, NULL) == ARG
    assert w(P, P, P, P, P, 1, 0, 4096, 256, 256, P, need - 1, NULL) == ARG
    assert w(P, P, P, P, P, 1, 0, 4096, 256, 256, ODD, need, NULL) == ALIGN
    need = lib.dg_fp8_dgrad_workspace(16, 4096, 4096)
    assert need >= 2 * 16 * 4096 * 4 and lib.dg_fp8_dgrad_workspace(16, 0, 4096) == 0
    assert d(P, P, P, P, P, 16, 4096, 4096, NULL, 0, NULL) == ARG
    assert d(P, P, P, P, P, 16, 4096, 4096, ODD, need, NULL) == ALIGN
    gd = lib.dg_fp8_grouped_dgrad_contiguous
    assert gd(P, P, P, P, P, P, 100, 2, 128, 128, NULL) == SHAPE
    assert gd(P, P, P, P, P, P, 128, 2, 64, 128, NULL) == SHAPE        # N % 128
    assert gd(P, P, P, P, P, P, 128, 1025, 128, 128, NULL) == SHAPE
    assert gd(P, P, P, P, P, NULL, 128, 2, 128, 128, NULL) == ARG
    assert gd(P, P, P, P, P, ODD, 128, 2, 128, 128, NULL) == ALIGN
    gw = lib.dg_fp8_grouped_wgrad_contiguous
    assert gw(P, P, P, P, P, 1, 0, P, 128, 2, 64, 128, NULL) == SHAPE
    assert gw(P, P, P, P, P, 0, 1, P, 128, 2, 128, 128, NULL) == ARG
    assert gw(P, P, P, P, P, 1, 0, NULL, 128, 2, 128, 128, NULL) == ARG
    assert gw(P, P, P, P, P, 1, 0, P, 128, 1 << 20, 1 << 20, 128, NULL) == SHAPE


def test_sizes_beyond_the_index_ranges_are_refused(lib):
    """Widths and products of sizes that 32 or 64 bits do not hold: refused before any of them is computed with."""
    for H in (1 << 31, 1 << 53, (1 << 63) - 16):
        assert lib.dg_moe_dispatch_quantize(P, NULL, P, P, 8, 2, H, 128, 4, P, P, NULL, 0, NULL) == SHAPE
        assert lib.dg_moe_dispatch_quantize_masked(P, P, P, 8, 2, H, 4, 64, P, P, NULL) == SHAPE
        assert lib.dg_moe_combine(P, P, P, 1 << 29, 2, H, 128, P, NULL) == SHAPE
        assert lib.dg_moe_combine_backward(P, P, P, 8, 2, H, 128, P, NULL) == SHAPE
    for N in (1 << 31, 1 << 54, 1 << 62):  # 1024 * 2^54 is 0 in 64 bits
        assert lib.dg_fp8_grouped_dgrad_contiguous(P, P, P, P, P, P, 128, 1024, N, 128, NULL) == SHAPE
        assert lib.dg_fp8_grouped_wgrad_contiguous(P, P, P, P, P, 1, 0, P, 128, 1024, N, 128, NULL) == SHAPE
        assert lib.dg_fp8_dgrad_blockscaled(P, P, P, P, P, 8, N, 128, NULL, 0, NULL) == SHAPE
        assert lib.dg_swiglu_quantize(P, NULL, 0, 8, N, P, P, NULL, NULL, NULL) == SHAPE


def test_binding_refuses_host_tensors(lib):
    """Types, ranks and devices are checked before the library sees an address."""
    with pytest.raises(ValueError):
        binding.moe_sort(torch.zeros((4, 2), dtype=torch.int32), 4)
    with pytest.raises(ValueError):
        binding.swiglu_quantize(torch.zeros((4, 256), dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        binding.moe_combine(torch.zeros((4, 16), dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32))
