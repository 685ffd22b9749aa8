"""GPU checks of the 16-bit experts at ends of their documented range, beside
tests/test_gpu_dense.py (whose bounds they use)."""
import numpy as np
import pytest
import torch

import quantized_moe_expert_top_amd as q
from tests.test_gpu_dense import DEV, KERNELS, bound, close, f64, i32, tile

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kernel", KERNELS)
def test_weights_just_below_4_gib(lib, kernel):
    """2040 channels of 2^20 inputs: offsets of the last rows fill 32 bits, those of rows past them would not fit."""
    N, K, M = 2040, 1 << 20, 3
    g = torch.Generator(device=DEV).manual_seed(1)
    w = torch.empty(1, N, K, dtype=torch.bfloat16, device=DEV)
    for n in range(0, N, 255):
        w[0, n:n + 255] = torch.randn(255, K, generator=g, device=DEV) / 1024
    a = torch.randn(M, K, generator=g, device=DEV).bfloat16()
    seg, kr = i32([0, M]), KERNELS[kernel]
    at = [0, 1, 31, 1000, 2016, 2032, 2039]
    got = q.moe_grouped_gemm(w, a, seg, M, q.MOE_EPI_NONE_F32, kernel=kr)
    some = f64(w[0, at])
    ref, mag = f64(a) @ some.T, np.abs(f64(a)) @ np.abs(some).T
    close(f64(got[:, at]), ref, bound(ref, mag, K, "fp32"))
    assert torch.isfinite(got).all()
    pairs = i32([2, 0, 1])
    assert torch.equal(q.moe_grouped_gemm(w, a, seg, M, q.MOE_EPI_NONE_F32, gather_pair=pairs, kernel=kr), got[[2, 0, 1]])
    dy = torch.randn(M, N, generator=g, device=DEV).bfloat16()
    da = q.moe_grouped_gemm_grad_rows(w, dy, seg, M, q.MOE_EPI_NONE_F32, kernel=kr)
    cols = [0, 7, 63, 1 << 19, K - 65, K - 1]
    some = f64(w[0][:, cols])
    ref, mag = f64(dy) @ some, np.abs(f64(dy)) @ np.abs(some)
    close(f64(da[:, cols]), ref, bound(ref, mag, N, "fp32"))
    dw = q.moe_grouped_gemm_grad_weights(dy, a, seg, 1, M, q.MOE_EPI_NONE, kernel=tile(kr))
    ref = f64(dy[:, at]).T @ f64(a[:, cols])
    mag = np.abs(f64(dy[:, at])).T @ np.abs(f64(a[:, cols]))
    close(f64(dw[0][at][:, cols]), ref, bound(ref, mag, M, "bf16"))
