"""GPU checks of the 16-bit experts at ends of their documented range, beside
tests/test_gpu_dense.py (whose bounds they use)."""
import numpy as np
import pytest
import torch

import quantized_moe_expert_top_amd as q
from oracle import dense_oracle as do
from tests.test_gpu_dense import DEV, DT, EPI, KERNELS, Batch, bound, close, f64, i32, tile

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


def layer(seed, T, E, k, H, I, dt, size=1.0):
    r = np.random.default_rng(seed)
    mk = lambda *s: torch.from_numpy(r.standard_normal(s)).to(DEV)  # noqa: E731
    return (mk(T, H).to(dt), mk(T, E).float(), (mk(E, 2 * I, H) / H ** 0.5 * size).to(dt),
            (mk(E, H, I) / I ** 0.5).to(dt), mk(T, H).bfloat16())


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,E,k,H,I", [(3, 4, 3, 64, 32), (70, 12, 8, 136, 48)])
def test_shares_of_dx_are_added_unrounded(lib, dt, T, E, k, H, I):
    """dx rounds once: the k experts' fp32 shares, added in fp32 in the slots' order, to bf16."""
    x, logits, gu, dn, dout = layer(1, T, E, k, H, I, dt)
    buf = q.moe_expert_layer_forward(x, logits, k, gu, dn, keep=True)
    g = q.moe_expert_layer_backward(dout, x, gu, dn, buf)
    p, P = buf.perm, T * k
    c = q.moe_unpermute_combine_grad(dout, buf.y_perm, p.pair_pos, buf.w, T, k, dtype=dt)
    dpre = q.moe_grouped_gemm_grad_rows(dn, c.dy, p.seg_offsets, P, q.MOE_EPI_SWIGLU_GRAD, pre=buf.pre)
    share = q.moe_grouped_gemm_grad_rows(gu, dpre, p.seg_offsets, P, q.MOE_EPI_NONE_F32)
    ref = f64(share)[p.pair_pos.cpu().numpy().reshape(T, k)]
    # an fp32 addition is off by 2^-24 of each partial sum; bf16 rounds once, to at most half a step
    mag = np.abs(ref).sum(1)
    close(f64(g.dx), ref.sum(1), 2.0 ** -8 * np.abs(ref.sum(1)) + (1 + 2.0 ** -8) * k * 2.0 ** -24 * mag)


def test_shares_of_dx_past_fp16s_range(lib):
    """Shares of dx above 65504, dx itself in bf16: finite, near the float64 gradient."""
    T, E, k, H, I = 6, 2, 2, 64, 32
    x, logits, gu, dn, dout = layer(2, T, E, k, H, I, torch.float16, size=64.0)
    x = x / 64
    dout = (dout.float() * 2048).bfloat16()
    buf = q.moe_expert_layer_forward(x, logits, k, gu, dn, keep=True)
    g = q.moe_expert_layer_backward(dout, x, gu, dn, buf)
    v = x.double().cpu().requires_grad_()
    gate = torch.softmax(logits.double().cpu().gather(1, buf.ids.long().cpu()), -1)
    rows = []
    for t in range(T):
        s = 0.0
        for j in range(k):
            e = int(buf.ids[t, j])
            y = gu[e].double().cpu() @ v[t]
            s = s + gate[t, j] * (dn[e].double().cpu() @ (torch.nn.functional.silu(y[:I]) * y[I:]))
        rows.append(s)
    (torch.stack(rows) * dout.double().cpu()).sum().backward()
    ref = v.grad.numpy()
    assert np.abs(ref).max() > 2 * 65504
    # roundings of h, y, dy, pre (its effect at most doubled) and dpre to fp16, of dx to bf16, in L2
    assert np.linalg.norm(f64(g.dx) - ref) <= (6 * 2.0 ** -11 + 2.0 ** -8) * np.linalg.norm(ref)


@pytest.mark.parametrize("counts,N,K", [([5000], 64, 40), ([0, 2100, 1030], 72, 136), ([2300, 1], 16, 264)])
@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_split_rows_in_every_type(lib, dt, out, counts, N, K):
    """The weights' gradient of long segments of few weights: fp32 parts in the workspace, added and rounded once by a
    second kernel, for either operand type and every output type."""
    n = np.array(counts).reshape(-1, 1, 1)
    for gather in (False, True):
        b = Batch(11, counts, N, K, dt, k=2 if gather else 1, gather=gather)
        ref, mag = do.grad_weights(f64(b.dy), b.rows, b.offsets)
        for kernel in (q.MOE_KERNEL_AUTO, q.MOE_KERNEL_TILE128):
            need = q.moe_grouped_gemm_grad_weights_workspace_size(b.E, N, K, b.M, kernel)
            assert need >= 2 * b.E * N * K * 4  # split
            ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)  # NaNs
            got = q.moe_grouped_gemm_grad_weights(b.dy, b.a, b.seg, b.E, b.M, EPI[out], gather_pair=b.pairs, k=b.k,
                                                  kernel=kernel, workspace=ws)
            assert got.dtype == DT[out]
            close(f64(got), ref, bound(ref, mag, n, out), f"gather {gather}")


@pytest.mark.parametrize("kernel", KERNELS)
def test_layer_with_every_kernel_choice(lib, kernel):
    """Forward and backward by one choice each: the gradients of a choice differ from AUTO's by the sums' order alone."""
    T, E, k, H, I = 40, 5, 2, 72, 40
    x, logits, gu, dn, dout = layer(3, T, E, k, H, I, torch.bfloat16)
    want = q.moe_expert_layer_forward(x, logits, k, gu, dn, keep=True)
    ref = q.moe_expert_layer_backward(dout, x, gu, dn, want)
    buf = q.moe_expert_layer_forward(x, logits, k, gu, dn, keep=True, kernel=KERNELS[kernel])
    got = q.moe_expert_layer_backward(dout, x, gu, dn, buf, kernel=KERNELS[kernel])
    # an fp32 sum of another order may round a 16-bit value the other way, a whole step (2^-7), at most
    for a, b in ((buf.out, want.out), (got.dx, ref.dx), (got.dgate_up, ref.dgate_up), (got.ddown, ref.ddown)):
        assert torch.linalg.vector_norm(a.double() - b.double()) <= 2.0 ** -7 * torch.linalg.vector_norm(b.double())
