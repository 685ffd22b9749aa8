"""Experts in 16 bits and low-rank adapters without a GPU: the float64
references against hand-computed values and differences, the C entry points'
refusals (before any device call), the binding's own checks, and the host
layer under sanitizers."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import quantized_moe_expert_top_amd as q
from oracle import dense_oracle as do

OK, NULL_ARG, BAD_SHAPE, BAD_FORMAT, MISALIGNED, WS_SMALL, UNSUPPORTED, HIP = range(8)
A, B, C, D = (ctypes.c_void_p(v) for v in (0x1000, 0x2000, 0x3000, 0x4000))
ODD = ctypes.c_void_p(0x1008)
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    return q.lib()


# ------------------------------------------------------------------ references
def test_reference_product_by_hand():
    w = np.array([[[1.0, 2.0], [0.0, -1.0]], [[3.0, 0.0], [1.0, 1.0]]])
    a = np.array([[1.0, 1.0], [2.0, 0.0], [0.0, 5.0]])
    y, m = do.product(w, a, [0, 1, 3])
    assert y.tolist() == [[3, -1], [6, 2], [0, 5]] and m.tolist() == [[3, 1], [6, 2], [0, 5]]
    dw, _ = do.grad_weights(y, a, [0, 1, 1, 3])
    assert dw[1].tolist() == [[0, 0], [0, 0]] and dw[0].tolist() == [[3, 3], [-1, -1]]
    assert dw[2].tolist() == [[12, 0], [4, 25]]


def test_reference_gradients_by_differences():
    r = np.random.default_rng(0)
    w, a, c = r.standard_normal((2, 6, 4)), r.standard_normal((5, 4)), r.standard_normal((5, 3))
    off = [0, 2, 5]
    loss = lambda w, a: (do.swiglu(do.product(w, a, off)[0]) * c).sum()  # noqa: E731
    dpre = do.swiglu_grad(c, do.product(w, a, off)[0])
    da, dw = do.grad_rows(w, dpre, off)[0], do.grad_weights(dpre, a, off)[0]
    h = 1e-6
    for x, g, f in ((a, da, lambda v: loss(w, v)), (w, dw, lambda v: loss(v, a))):
        for _ in range(6):
            d = r.standard_normal(x.shape)
            assert abs((f(x + h * d) - f(x - h * d)) / (2 * h) - (g * d).sum()) < 1e-6 * (1 + abs((g * d).sum()))


def test_reference_adapters_and_combine_by_hand():
    y, x = np.zeros((3, 2)), np.array([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]])
    out, _ = do.adapters(y, x, np.ones((1, 1, 2)), np.array([[[1.0], [-2.0]]]), [0, -1, 1], [0.5])
    assert out.tolist() == [[1.5, -3], [0, 0], [0, 0]]
    dy, dw, _, dl = do.combine_grad(np.array([[2.0, 1.0]]), np.array([[1.0, 0.0], [0.0, 3.0]]), np.array([[1, 0]]),
                                    np.array([[0.25, 0.75]]), 2, np.array([[4, 1]]), 5)
    assert dy.tolist() == [[1.5, 0.75], [0.5, 0.25]] and dw.tolist() == [[3, 2]]
    assert dl.tolist() == [[0, -0.1875, 0, 0, 0.1875]]


# -------------------------------------------------------------------- refusals
def gemm(lib, w=A, dtype=0, E=4, N=32, K=64, a=B, rows=10, gather=None, k=1, seg=C, M=10, epi=0, kernel=0, pre=None, out=D):
    return lib.moe_grouped_gemm(w, dtype, E, N, K, a, rows, gather, k, seg, M, epi, kernel, pre, out, None)


def test_product_refusals(lib):
    for kw in (dict(M=0), dict(M=0, w=None, a=None, seg=None, out=None)):
        assert gemm(lib, **kw) == OK
    for want, cases in (
            (BAD_FORMAT, [dict(dtype=1), dict(dtype=7), dict(epi=4), dict(epi=6), dict(epi=-1), dict(kernel=10), dict(kernel=-1),
                          dict(pre=ctypes.c_void_p(0x9000))]),
            (BAD_SHAPE, [dict(E=0), dict(E=1025), dict(N=0), dict(K=0), dict(M=-1), dict(rows=9), dict(rows=-1),
                         dict(gather=A, k=0), dict(gather=A, k=1, rows=9), dict(out=A), dict(out=B),
                         dict(epi=1, pre=B), dict(epi=1, pre=D)]),
            (UNSUPPORTED, [dict(N=12), dict(K=20), dict(N=24, epi=1), dict(kernel=3), dict(kernel=8), dict(N=(1 << 20) + 8),
                           dict(K=(1 << 20) + 8), dict(N=1 << 16, K=1 << 15), dict(gather=A, rows=1 << 25, K=64, k=1),
                           dict(M=1 << 30, rows=1 << 30)]),
            (NULL_ARG, [dict(w=None), dict(a=None), dict(seg=None), dict(out=None)]),
            (MISALIGNED, [dict(w=ODD), dict(a=ODD), dict(out=ODD), dict(seg=ctypes.c_void_p(0x3002)),
                          dict(gather=ctypes.c_void_p(0x3002), k=1), dict(epi=1, pre=ODD)])):
        for kw in cases:
            assert gemm(lib, **kw) == want, (want, kw)
            assert lib.moe_last_error_detail()


def rows(lib, w=A, dtype=0, E=4, N=32, K=64, dy=B, seg=C, M=10, epi=0, kernel=0, pre=None, out=D):
    return lib.moe_grouped_gemm_grad_rows(w, dtype, E, N, K, dy, seg, M, epi, kernel, pre, out, None)


def test_grad_rows_refusals(lib):
    assert rows(lib, M=0) == OK
    for want, cases in (
            (BAD_FORMAT, [dict(dtype=1), dict(epi=1), dict(epi=5), dict(kernel=99)]),
            (BAD_SHAPE, [dict(E=0), dict(M=-1), dict(out=A), dict(out=B), dict(epi=6, pre=D)]),
            (UNSUPPORTED, [dict(N=12), dict(K=12), dict(kernel=4), dict(M=1 << 30)]),
            (NULL_ARG, [dict(w=None), dict(dy=None), dict(seg=None), dict(out=None), dict(epi=6), dict(pre=A)]),
            (MISALIGNED, [dict(w=ODD), dict(dy=ODD), dict(out=ODD), dict(epi=6, pre=ODD)])):
        for kw in cases:
            assert rows(lib, **kw) == want, (want, kw)


def weights(lib, dy=A, a=B, dtype=0, E=4, N=32, K=64, A_rows=10, gather=None, k=1, seg=C, M=10, epi=2, kernel=0, out=D, ws=None,
            ws_bytes=0):
    return lib.moe_grouped_gemm_grad_weights(dy, a, dtype, E, N, K, A_rows, gather, k, seg, M, epi, kernel, out, ws, ws_bytes,
                                             None)


def test_grad_weights_refusals(lib):
    for want, cases in (
            (BAD_FORMAT, [dict(dtype=1), dict(epi=1), dict(epi=6), dict(kernel=99)]),
            (BAD_SHAPE, [dict(E=0), dict(M=-1), dict(A_rows=9), dict(gather=A, k=0), dict(out=A), dict(out=B)]),
            (UNSUPPORTED, [dict(N=12), dict(K=12), dict(kernel=1), dict(kernel=6), dict(gather=A, A_rows=1 << 25)]),
            (NULL_ARG, [dict(dy=None), dict(a=None), dict(seg=None), dict(out=None), dict(out=None, M=0)]),
            (MISALIGNED, [dict(dy=ODD), dict(a=ODD), dict(out=ODD)])):
        for kw in cases:
            assert weights(lib, **kw) == want, (want, kw)
    size = lib.moe_grouped_gemm_grad_weights_workspace_size
    need = size(1, 64, 40, 5000, 0)
    assert need > 0 and need % (64 * 40 * 4) == 0
    long = dict(E=1, N=64, K=40, M=5000, A_rows=5000)
    assert weights(lib, **long) == WS_SMALL and weights(lib, **long, ws=A, ws_bytes=need - 1) == WS_SMALL
    assert weights(lib, **long, ws=ODD, ws_bytes=need) == MISALIGNED
    assert size(1, 64, 40, 5000, 9) == 0 and size(64, 2048, 2048, 65536, 0) == 0
    assert size(0, 64, 40, 1, 0) == 0 and size(1, 12, 40, 1, 0) == 0 and size(1, 64, 40, -1, 0) == 0 and size(1, 64, 40, 9, 1) == 0


def combine(lib, dout=A, y=B, y_dtype=2, pos=C, nv=None, w=D, ids=None, T=4, k=2, H=64, E=8, dy_dtype=0,
            dy=ctypes.c_void_p(0x5000), dw=ctypes.c_void_p(0x6000), dl=None):
    return lib.moe_unpermute_combine_grad(dout, y, y_dtype, pos, nv, w, ids, T, k, H, E, dy_dtype, dy, dw, dl, None)


def test_combine_grad_refusals(lib):
    assert combine(lib, T=0) == OK
    for want, cases in (
            (BAD_FORMAT, [dict(y_dtype=3), dict(dy_dtype=1), dict(dy_dtype=9)]),
            (BAD_SHAPE, [dict(T=-1), dict(T=1 << 24), dict(k=0), dict(k=1025), dict(T=(1 << 24) - 1, k=1024), dict(H=0),
                         dict(H=12), dict(ids=A, dl=B, E=0), dict(ids=A, dl=B, E=1025), dict(dy=A), dict(dy=B), dict(dw=D),
                         dict(ids=A, dl=ctypes.c_void_p(0x6000))]),
            (NULL_ARG, [dict(dout=None), dict(y=None), dict(pos=None), dict(dy=None), dict(dw=None), dict(ids=A),
                        dict(dl=A), dict(ids=A, dl=B, w=None)]),
            (MISALIGNED, [dict(dout=ODD), dict(y=ODD), dict(dy=ODD), dict(dw=ctypes.c_void_p(0x6002))])):
        for kw in cases:
            assert combine(lib, **kw) == want, (want, kw)


def adapters(lib, y=A, y_dtype=0, x=B, a=C, b=D, dtype=0, scale=None, n=3, r=16, K=64, N=32, seg=ctypes.c_void_p(0x7000),
             rows=ctypes.c_void_p(0x8000), T=5, out=ctypes.c_void_p(0x9000)):
    return lib.moe_adapter_add(y, y_dtype, x, a, b, dtype, scale, n, r, K, N, seg, rows, T, out, None)


def test_adapter_refusals(lib):
    assert adapters(lib, T=0) == OK
    for want, cases in (
            (BAD_FORMAT, [dict(y_dtype=3), dict(dtype=1)]),
            (BAD_SHAPE, [dict(n=0), dict(n=1025), dict(T=-1), dict(T=1 << 24), dict(r=0), dict(K=0), dict(N=0), dict(out=B),
                         dict(out=C), dict(out=D)]),
            (UNSUPPORTED, [dict(r=4), dict(r=136), dict(K=60), dict(N=12), dict(T=1 << 23, K=1 << 10),
                           dict(n=1024, r=128, K=1 << 15), dict(n=1024, r=128, N=1 << 15)]),
            (NULL_ARG, [dict(y=None), dict(x=None), dict(a=None), dict(b=None), dict(seg=None), dict(rows=None),
                        dict(out=None)]),
            (MISALIGNED, [dict(y=ODD), dict(x=ODD), dict(a=ODD), dict(b=ODD), dict(out=ODD),
                          dict(scale=ctypes.c_void_p(0x7002)), dict(rows=ctypes.c_void_p(0x7002))])):
        for kw in cases:
            assert adapters(lib, **kw) == want, (want, kw)


# --------------------------------------------------------- the binding's checks
def test_binding_refuses(lib):
    """What would send a kernel past a tensor is refused before the library is called."""
    bf, i = torch.bfloat16, torch.int32
    w, a, seg = torch.zeros(2, 32, 16, dtype=bf), torch.zeros(6, 16, dtype=bf), torch.zeros(3, dtype=i)
    dy = torch.zeros(6, 32, dtype=bf)
    for call, what in (
            (lambda: q.moe_grouped_gemm(w.float(), a, seg, 6), "bfloat16 or float16"),
            (lambda: q.moe_grouped_gemm(w[0], a, seg, 6), "E"),
            (lambda: q.moe_grouped_gemm(w, a.half(), seg, 6), "A must be"),
            (lambda: q.moe_grouped_gemm(w, a, seg, 7), "A must be"),
            (lambda: q.moe_grouped_gemm(w, a[:, :8], seg, 6), "A must be"),
            (lambda: q.moe_grouped_gemm(w, a, seg[:2], 6), "seg_offsets"),
            (lambda: q.moe_grouped_gemm(w, a, seg.long(), 6), "seg_offsets"),
            (lambda: q.moe_grouped_gemm(w, a, seg, 6, gather_pair=seg), "gather_pair"),
            (lambda: q.moe_grouped_gemm(w, a, seg, 6, 6), "epilogue"),
            (lambda: q.moe_grouped_gemm(w, a, seg, 6, pre=dy), "pre goes with"),
            (lambda: q.moe_grouped_gemm(w, a, seg, 6, q.MOE_EPI_SWIGLU, pre=dy[:5]), "pre must be"),
            (lambda: q.moe_grouped_gemm(w, a, seg, 6), "GPU"),
            (lambda: q.moe_grouped_gemm_grad_rows(w, dy[:5], seg, 6), "dy must be"),
            (lambda: q.moe_grouped_gemm_grad_rows(w, dy, seg, 6, q.MOE_EPI_SWIGLU_GRAD), "needs pre"),
            (lambda: q.moe_grouped_gemm_grad_rows(w, dy, seg, 6, q.MOE_EPI_SWIGLU_GRAD, pre=a), "pre must be"),
            (lambda: q.moe_grouped_gemm_grad_rows(w, dy, seg, 6, q.MOE_EPI_SWIGLU), "epilogue"),
            (lambda: q.moe_grouped_gemm_grad_weights(dy, a[:5], seg, 2, 6), "A must be"),
            (lambda: q.moe_grouped_gemm_grad_weights(dy, a, seg, 3, 6), "seg_offsets"),
            (lambda: q.moe_grouped_gemm_grad_weights(dy, a, seg, 2, 6, q.MOE_EPI_SWIGLU), "epilogue"),
            (lambda: q.moe_unpermute_combine_grad(dy, dy, seg, None, 6, 1), "pair_pos"),
            (lambda: q.moe_unpermute_combine_grad(dy.half(), dy, seg, None, 6, 1), "dout"),
            (lambda: q.moe_unpermute_combine_grad(dy[:3], dy, torch.zeros(6, dtype=i), None, 3, 2, dtype=torch.float32), "dy in"),
            (lambda: q.moe_unpermute_combine_grad(dy[:3], dy, torch.zeros(6, dtype=i), None, 3, 2,
                                                  ids=torch.zeros(3, 2, dtype=i)), "topk_w"),
            (lambda: q.moe_adapter_add(dy, a, w[:, :8], w, seg, torch.zeros(6, dtype=i)), "B must be"),
            (lambda: q.moe_adapter_add(dy, a[:5], w[:, :8], torch.zeros(2, 32, 8, dtype=bf), seg, torch.zeros(6, dtype=i)), "x must"),
            (lambda: q.moe_adapter_add(dy, a, w[:, :8], torch.zeros(2, 32, 8, dtype=bf), seg, seg), "rows"),
            (lambda: q.moe_adapter_add(dy, a, w[:, :8], torch.zeros(2, 32, 8, dtype=bf), seg, torch.zeros(6, dtype=i),
                                       scale=torch.zeros(3)), "scale"),
            (lambda: q.moe_expert_layer_forward(a, torch.zeros(6, 2), 1, w, w), "do not fit"),
            (lambda: q.alloc_expert_layer(2, 2, 1, 16, 16, "cpu", dtype=torch.float32), "weights in")):
        with pytest.raises(ValueError, match=what):
            call()


def test_layer_buffers_must_fit(lib):
    bf = torch.bfloat16
    gu, dn = torch.zeros(2, 32, 16, dtype=bf), torch.zeros(2, 16, 16, dtype=bf)
    x, dout = torch.zeros(6, 16, dtype=bf), torch.zeros(6, 16, dtype=bf)
    buf = q.alloc_expert_layer(6, 2, 1, 16, 16, "cpu")
    with pytest.raises(ValueError, match="kept nothing"):
        q.moe_expert_layer_backward(dout, x, gu, dn, buf)
    with pytest.raises(ValueError, match="buffers of"):
        q.moe_expert_layer_backward(dout, x[:5], gu, dn, buf)
    with pytest.raises(ValueError, match="do not fit"):
        q.moe_expert_layer_backward(dout, x.half(), gu, dn, buf)
    kept = q.alloc_expert_layer(6, 2, 1, 16, 16, "cpu", keep=True)
    with pytest.raises(ValueError, match="gradients in"):
        q.moe_expert_layer_backward(dout, x, gu, dn, kept, grad_dtype=torch.float64)


def test_dense_host_layer_under_sanitizers(tmp_path):
    """abi_dense.cpp and its share of plan.cpp built for the CPU against stand-in launchers."""
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    csrc, here = os.path.join(ROOT, "quantized_moe_expert_top_amd", "csrc"), os.path.join(ROOT, "tests", "host_abi")
    exe = str(tmp_path / "dense_abi_test")
    subprocess.run([gxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-omit-frame-pointer",
                    "-fno-sanitize-recover=all", "-Wall", "-Wextra", "-Wno-unused-parameter", "-Werror",
                    "-I", os.path.join(ROOT, "include"), "-I", csrc, "-I", here,
                    *(os.path.join(csrc, f) for f in ("abi.cpp", "abi_dense.cpp", "plan.cpp")),
                    *(os.path.join(here, f) for f in ("stub_device.cpp", "dense_abi_test.cpp")), "-o", exe, "-pthread"],
                   check=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "dense host layer checks passed" in r.stdout


def test_readme_shows_the_tested_calls():
    from tests.test_gpu_dense import README_CALLS
    assert "```\n" + README_CALLS + "```" in open(os.path.join(ROOT, "README.md")).read()
