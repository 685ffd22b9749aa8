"""Limits of the 16-bit products' calls that are checked on the host, without
a GPU."""
import ctypes

import pytest

import quantized_moe_expert_top_amd as q

UNSUPPORTED = 6
W, A, SEG, OUT = (ctypes.c_void_p(v) for v in (0x1000, 0x2000, 0x3000, 0x4000))


@pytest.fixture(scope="module")
def lib():
    return q.lib()


def product(lib, E, N, K, M, kernel):
    return lib.moe_grouped_gemm(W, 0, E, N, K, A, M, None, 1, SEG, M, q.MOE_EPI_NONE, kernel, None, OUT, None)


def rows(lib, E, N, K, M, kernel):
    return lib.moe_grouped_gemm_grad_rows(W, 0, E, N, K, A, SEG, M, q.MOE_EPI_NONE, kernel, None, OUT, None)


@pytest.mark.parametrize("call,N,K,width", [(product, 8, 16, 1), (product, 1 << 20, 8, 1 << 15), (rows, 16, 8, 1),
                                            (rows, 8, 1 << 20, 1 << 14)])
@pytest.mark.parametrize("E", [1, 1024])
def test_small_kernel_refuses_more_workgroups_than_a_launch_holds(lib, call, N, K, width, E):
    """One of 256 threads per 32 rows (a segment's last may be partial) and 32 columns (by the rows 64): 2^24 are 2^32
    threads.  The refusal comes before any device call, names the limit, and is MOE_KERNEL_SMALL's alone."""
    workgroups = lambda M: (M // 32 + min(M, E)) * width  # noqa: E731
    fits, refused = 0, (1 << 30) - 1  # grows with M: between the two lies the last that fits
    while refused - fits > 1:
        M = (fits + refused) // 2
        fits, refused = (M, refused) if workgroups(M) < 1 << 24 else (fits, M)
    for M in (refused, (1 << 30) - 1):
        assert call(lib, E, N, K, M, q.MOE_KERNEL_SMALL) == UNSUPPORTED
        assert b"2^24" in lib.moe_last_error_detail()
        assert call(lib, E, N, K, M, q.MOE_KERNEL_TILE128) != UNSUPPORTED
    assert fits > 0 and call(lib, E, N, K, fits, q.MOE_KERNEL_SMALL) != UNSUPPORTED
