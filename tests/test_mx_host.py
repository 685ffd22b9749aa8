"""Scored routing and MX path without a GPU: the float64 references against
hand-computed values, the C entry points' refusals (before any device call)
and the binding's own checks."""
import ctypes

import numpy as np
import pytest
import torch

import quantized_moe_expert_top_amd as q
from oracle import mx_oracle as mx

OK, NULL_ARG, BAD_SHAPE, BAD_FORMAT, MISALIGNED, WS_SMALL, UNSUPPORTED, HIP = range(8)
A = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1002)


@pytest.fixture(scope="module")
def lib():
    return q.lib()


# ------------------------------------------------------------------ references
def test_reference_tables():
    assert mx.TABLE[mx.E2M1].tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    t = mx.TABLE[mx.E4M3]
    assert t[-1] == 448 and t[1] == 2.0 ** -9 and t[8] == 2.0 ** -6 and (np.diff(t) > 0).all()


@pytest.mark.parametrize("fmt,top", [(mx.E4M3, 448.0), (mx.E2M1, 6.0)])
def test_reference_scale(fmt, top):
    """The scale is the smallest power of two at which the largest magnitude fits."""
    m = np.array([top, np.nextafter(np.float32(top), np.float32(1e9)), top / 2, 1.0, 2.0 ** -126, 1e-45, 3.4028235e38, 0.0])
    p = mx.scale_exponent(m, fmt).astype(np.float64)
    assert (m <= top * np.exp2(p)).all()
    assert ((m > top * np.exp2(p - 1)) | (p == -126)).all()
    assert p[0] == 0 and p[1] == 1 and p[2] == -1 and p[-1] == -126


def test_reference_rounding_ties():
    assert mx.nearest_code(np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]), mx.E2M1).tolist() == [0, 2, 2, 4, 4, 6, 6]
    x = np.zeros(32)
    x[:4] = [448, 17.0, 19.0, 2.0 ** -10]  # 16..32 in steps of 2; half the smallest element
    codes, scales = mx.quantize(x, mx.E4M3)
    assert mx.values(codes, scales, mx.E4M3)[:4].tolist() == [448, 16, 20, 0] and scales[0] == 127
    x[5] = np.inf
    codes, scales = mx.quantize(x, mx.E4M3)
    assert scales[0] == 255 and (codes == 0).all() and np.isnan(mx.values(codes, scales, mx.E4M3)).all()


def test_reference_routing_by_hand():
    ids, w = mx.route_scored([[0.0, 1.0, 2.0, 1.0]], 3)
    e = np.exp([2.0, 1.0, 1.0])
    assert ids.tolist() == [[2, 1, 3]] and np.allclose(w[0], e / e.sum())
    # two groups of two; sigmoid scores .5 .5 | .88 .12: by the best two 1.0 ties 1.0 up to rounding, by the best one group 1
    ids, w = mx.route_scored([[0.0, 0.0, 2.0, -2.0]], 2, sigmoid=True, n_group=2, group_top=1, renorm=False, scale=2.0)
    assert ids.tolist() == [[2, 3]] and np.allclose(w[0], 2 / (1 + np.exp([-2.0, 2.0])))
    ids, w = mx.route_scored([[0.0, -np.inf, np.nan, 1.0]], 3, bias=[0, 9, 9, -np.inf])
    assert ids.tolist() == [[0, -1, -1]] and w.tolist() == [[1, 0, 0]]


# -------------------------------------------------------------------- C refusals
def test_route_scored_validation(lib):
    def call(logits=A, bias=None, T=4, E=8, k=2, score=0, ng=1, tg=1, gt=1, scale=1.0, ids=A, w=A):
        return lib.moe_route_scored(logits, bias, T, E, k, score, ng, tg, gt, 1, scale, ids, w, None)
    assert call(T=-1) == call(E=0) == call(E=1025) == call(k=0) == call(k=9) == BAD_SHAPE
    assert call(T=1 << 28, E=1024, k=16) == call(T=1 << 25, k=1) == BAD_SHAPE
    assert call(score=2) == call(score=-1) == BAD_FORMAT
    assert call(ng=0) == call(ng=3) == call(E=1024, ng=128) == BAD_SHAPE
    assert call(ng=4, tg=5) == call(ng=4, tg=0) == call(gt=0) == call(gt=3) == BAD_SHAPE
    assert call(scale=float("nan")) == call(scale=float("inf")) == BAD_SHAPE
    assert call(logits=None) == call(ids=None) == call(w=None) == NULL_ARG
    assert call(logits=ODD) == call(bias=ODD) == call(ids=ODD) == call(w=ODD) == MISALIGNED
    assert call(T=0, logits=None, ids=None, w=None) == OK and lib.moe_last_error_detail() == b""


def test_mx_rows_validation(lib):
    B = ctypes.c_void_p(0x2000)

    def quant(x=B, dt=0, rows=4, K=64, fmt=1, c=A, s=A):
        return lib.moe_quantize_mx(x, dt, rows, K, fmt, c, s, None)

    def dequant(c=A, s=A, rows=4, K=64, fmt=1, dt=0, out=B):
        return lib.moe_dequantize_mx(c, s, rows, K, fmt, dt, out, None)
    for f in (quant, dequant):
        assert f(dt=3) == f(fmt=0) == f(fmt=3) == BAD_FORMAT
        assert f(rows=-1) == f(K=0) == f(K=48) == f(K=-32) == f(rows=1 << 36) == BAD_SHAPE
        assert f(c=None) == f(s=None) == NULL_ARG
        assert f(c=ctypes.c_void_p(0x1008)) == MISALIGNED
        assert f(rows=0, c=None, s=None) == OK
        assert f(c=B) == f(rows=(1 << 29), K=32) == BAD_SHAPE  # in place; 2^34 values
    assert quant(x=None) == dequant(out=None) == NULL_ARG
    assert quant(x=ctypes.c_void_p(0x1008)) == dequant(out=ctypes.c_void_p(0x1008)) == MISALIGNED


def test_rmsnorm_validation(lib):
    B, C, D, F = (ctypes.c_void_p(v) for v in (0x2000, 0x3000, 0x4000, 0x5000))

    def norm(x=A, r=B, w=C, dt=0, rows=4, H=64, eps=1e-5, sum=B, y=D, fmt=1, c=F, s=A):
        return lib.moe_rmsnorm_mx(x, r, w, dt, rows, H, eps, sum, y, fmt, c, s, None)
    assert norm(dt=3) == norm(fmt=3) == BAD_FORMAT
    assert norm(rows=-1) == norm(H=40) == norm(eps=-1.0) == norm(eps=float("nan")) == norm(eps=float("inf")) == BAD_SHAPE
    assert norm(H=16384 + 32) == UNSUPPORTED
    assert norm(x=None) == norm(w=None) == norm(r=None) == NULL_ARG            # sum without residual
    assert norm(c=None) == norm(s=None) == norm(fmt=0) == NULL_ARG             # codes exactly with a format
    assert norm(sum=None, y=None, fmt=0, c=None, s=None) == NULL_ARG           # no output
    assert norm(y=B) == BAD_SHAPE                                              # sum and y in one buffer
    assert norm(c=A) == norm(c=B) == norm(c=D) == norm(rows=1 << 24, H=32) == BAD_SHAPE     # codes over values; many rows
    assert norm(x=ctypes.c_void_p(0x1008)) == norm(w=ctypes.c_void_p(0x3008)) == norm(y=ctypes.c_void_p(8)) == MISALIGNED
    assert norm(rows=0, x=None, w=None) == OK


def mxdesc(layout=q.MOE_LAYOUT_TILED, E=4, N=128, K=256, codes=0x10000, scales=0x20000, version=q.MOE_ABI_VERSION):
    d = q.MxDesc()
    d.abi_version, d.layout, d.E, d.N, d.K, d.codes, d.scales = version, layout, E, N, K, codes, scales
    return d


def test_mx_weights_validation_and_sizes(lib):
    canon, tiled = q.MOE_LAYOUT_CANONICAL, q.MOE_LAYOUT_TILED
    fb = lambda d, f: lib.moe_mx_field_bytes(ctypes.byref(d), f)  # noqa: E731
    for layout in (canon, tiled):
        assert fb(mxdesc(layout), q.MOE_FIELD_CODES) == 4 * 128 * 256 // 2
        assert fb(mxdesc(layout), q.MOE_FIELD_SCALES) == 4 * 128 * 256 // 32
        assert fb(mxdesc(layout), q.MOE_FIELD_BASE) == 0
    assert fb(mxdesc(canon, K=384), q.MOE_FIELD_SCALES) == 4 * 128 * 12
    assert fb(mxdesc(tiled, K=384), q.MOE_FIELD_CODES) == 4 * 128 * 512 // 2
    assert fb(mxdesc(tiled, K=384), q.MOE_FIELD_SCALES) == 4 * 4 * 2 * 256   # padded to whole chunks of 256 inputs
    assert fb(mxdesc(N=48), q.MOE_FIELD_CODES) == fb(mxdesc(K=192), q.MOE_FIELD_CODES) == 0
    rep = lambda a, b: lib.moe_mx_repack(ctypes.byref(a), ctypes.byref(b), None)  # noqa: E731
    dst = mxdesc(codes=0x70000, scales=0x80000)
    assert rep(mxdesc(tiled), dst) == rep(mxdesc(canon), mxdesc(canon, codes=0x70000)) == BAD_FORMAT
    assert rep(mxdesc(canon, version=7), dst) == BAD_FORMAT
    assert rep(mxdesc(canon, N=256), dst) == rep(mxdesc(canon), mxdesc()) == BAD_SHAPE  # other sizes; in place
    assert rep(mxdesc(canon, codes=0), dst) == NULL_ARG
    assert rep(mxdesc(canon, codes=0x10008), dst) == rep(mxdesc(canon, scales=0x20002), dst) == MISALIGNED
    assert rep(mxdesc(canon, E=1025), mxdesc(E=1025)) == rep(mxdesc(canon, N=1 << 17, K=1 << 17), dst) == BAD_SHAPE
    big = dict(E=1024, N=1 << 13, K=1 << 14)  # 2^37 weights
    assert rep(mxdesc(canon, codes=0x30000, scales=0x40000, **big), mxdesc(**big)) == BAD_SHAPE


def test_grouped_mxgemm_validation(lib):
    def gemm(d=None, a=A, s=A, fmt=1, rows=64, gather=A, k=2, seg=A, M=128, epi=q.MOE_EPI_NONE, kernel=0, out=ctypes.c_void_p(0x2000),
             osc=None):
        d = d or mxdesc()
        return lib.moe_grouped_mxgemm(ctypes.byref(d), a, s, fmt, rows, gather, k, seg, M, epi, kernel, out, osc, None)
    assert gemm(mxdesc(q.MOE_LAYOUT_CANONICAL)) == gemm(mxdesc(version=2)) == gemm(fmt=0) == gemm(epi=6) == BAD_FORMAT
    assert gemm(epi=-1) == gemm(kernel=10) == gemm(kernel=-1) == BAD_FORMAT
    assert gemm(kernel=q.MOE_KERNEL_LDS_DMA) == gemm(kernel=q.MOE_KERNEL_SMALL_PER_WIDTH) == UNSUPPORTED
    assert gemm(fmt=2, kernel=q.MOE_KERNEL_TILE64_SPLIT_K) == UNSUPPORTED       # K = 256
    assert gemm(mxdesc(K=512), kernel=q.MOE_KERNEL_TILE64_SPLIT_K) == UNSUPPORTED  # e4m3 rows
    assert gemm(mxdesc(N=96), epi=q.MOE_EPI_SWIGLU) == gemm(mxdesc(N=48)) == gemm(mxdesc(K=160)) == UNSUPPORTED
    assert gemm(M=-1) == gemm(rows=-1) == gemm(k=0) == gemm(rows=63) == gemm(gather=None, rows=127) == BAD_SHAPE
    assert gemm(out=A) == BAD_SHAPE                                             # in place
    assert gemm(a=None) == gemm(s=None) == gemm(seg=None) == gemm(out=None) == NULL_ARG
    assert gemm(osc=A) == gemm(epi=q.MOE_EPI_SWIGLU_E4M3) == NULL_ARG           # scales exactly with an MX epilogue
    assert gemm(a=ctypes.c_void_p(0x1008)) == gemm(out=ctypes.c_void_p(0x1008)) == MISALIGNED
    assert gemm(s=ODD) == gemm(seg=ODD) == gemm(gather=ODD) == MISALIGNED
    assert gemm(mxdesc(K=1 << 20), rows=1 << 12) == UNSUPPORTED                 # 4 GiB of activation codes
    assert gemm(M=0, a=None, s=None, seg=None, out=None) == OK


def test_mx_layer_validation(lib):
    def call(**kw):
        gu = mxdesc(E=4, N=2 * kw.pop("I", 256), K=kw.get("H", 128))
        dn = mxdesc(E=kw.pop("E_down", 4), N=kw.pop("N_down", kw.pop("H", 128)), K=256)
        f = dict(abi_version=q.MOE_ABI_VERSION, T=3, k=2, x_dtype=q.MOE_DTYPE_BF16, x_fmt=1, h_fmt=1, y_dtype=q.MOE_DTYPE_F16,
                 kernel=0, score=0, n_group=1, topk_group=1, group_top=1, renormalize=1, scale=1.0, bias=None,
                 workspace_bytes=512, gate_up=ctypes.pointer(gu), down=ctypes.pointer(dn))
        for i, n in enumerate(("x", "logits", "topk_ids", "topk_w", "expert_counts", "seg_offsets", "sorted_pair", "pair_pos", "workspace",
                  "x_codes", "x_scales", "h_codes", "h_scales", "y", "out")):
            f[n] = 0x1000 * (i + 1)
        f.update(kw)
        layer = q.MxLayer()
        for n, v in f.items():
            setattr(layer, n, v)
        return lib.moe_mx_layer(ctypes.byref(layer), None)
    assert lib.moe_mx_layer(None, None) == NULL_ARG
    assert call(abi_version=2) == call(x_dtype=5) == call(x_fmt=0) == call(h_fmt=3) == call(y_dtype=3) == BAD_FORMAT
    assert call(score=2) == call(kernel=10) == BAD_FORMAT
    assert call(kernel=6) == call(kernel=q.MOE_KERNEL_TILE64_SPLIT_K) == UNSUPPORTED  # I = 256
    assert call(I=320) == call(E_down=5) == call(N_down=256) == BAD_SHAPE            # the two products do not fit
    assert call(T=-1) == call(k=5) == call(n_group=3) == call(scale=float("nan")) == BAD_SHAPE
    for n in ("logits", "topk_ids", "topk_w", "expert_counts", "seg_offsets", "sorted_pair", "pair_pos", "workspace",
              "x_codes", "x_scales", "h_codes", "h_scales", "y", "out"):
        assert call(**{n: None}) == NULL_ARG, n
    assert call(workspace_bytes=511) == WS_SMALL
    for a, b in (("x", "x_codes"), ("x_codes", "h_codes"), ("h_codes", "y"), ("y", "out")):
        assert call(**{a: 0x100000, b: 0x100000}) == BAD_SHAPE, (a, b)
    size = lib.moe_mx_layer_workspace_size
    assert size(3, 2, 4) == 256 + 256                       # the flag words; one chunk of 16 tokens, 5 counters
    assert size(16384, 8, 64) == 256 + 1024 * 65 * 4        # 1024 chunks
    assert size(131072, 8, 64) == 256 + 8192 * 65 * 4       # not more than 3 counters per pair
    assert size(131072, 1, 64) == lib.moe_permute_workspace_size(131072, 1, 64, 1)
    assert size(-1, 2, 4) == size(3, 0, 4) == size(3, 2, 1025) == size(1 << 28, 16, 64) == 0
    for n in ("x", "x_codes", "h_codes", "y", "out", "workspace"):
        assert call(**{n: 0x1008}) == MISALIGNED, n
    for n in ("x_scales", "h_scales", "logits", "bias", "seg_offsets", "sorted_pair", "pair_pos", "expert_counts"):
        assert call(**{n: 0x1002}) == MISALIGNED, n
    assert call(T=0, logits=None, x=None, out=None) == OK


# ------------------------------------------------------------ the binding's checks
def test_mx_rows_object():
    u8 = dict(dtype=torch.uint8)
    r = q.MxRows(torch.zeros((3, 64), **u8), torch.zeros((3, 4), **u8), q.MOE_MX_E2M1)
    assert r.K == 128 and r.shape == (3, 128)
    for codes, scales, fmt in (((3, 64), (3, 4), q.MOE_MX_E4M3), ((3, 64), (2, 2), q.MOE_MX_E4M3), ((3, 64), (3, 2), 7)):
        with pytest.raises(ValueError):
            q.MxRows(torch.zeros(codes, **u8), torch.zeros(scales, **u8), fmt)
    with pytest.raises(ValueError):
        q.MxRows(torch.zeros((3, 64), dtype=torch.int8), torch.zeros((3, 2), **u8), q.MOE_MX_E4M3)
    with pytest.raises(ValueError):
        q.alloc_mx_rows((4, 40), q.MOE_MX_E4M3, "cpu")
    assert q.alloc_mx_rows((2, 3, 64), q.MOE_MX_E2M1, "cpu").codes.shape == (2, 3, 32)


def test_binding_refuses_host_and_odd_tensors():
    x = torch.zeros(4, 64)
    for call in (lambda: q.moe_quantize_mx(x), lambda: q.moe_rmsnorm_mx(x, torch.ones(64), 1e-5),
                 lambda: q.moe_route_scored(x, 2),
                 lambda: q.moe_dequantize_mx(q.alloc_mx_rows((4, 64), q.MOE_MX_E4M3, "cpu"))):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(ValueError):
        q.moe_quantize_mx(x.double())
    with pytest.raises(ValueError, match="bias"):
        q.moe_route_scored(x, 2, bias=torch.zeros(63))
    with pytest.raises(ValueError, match="weight"):
        q.moe_rmsnorm_mx(x, torch.ones(32), 1e-5)
    with pytest.raises(ValueError, match="sum without residual"):
        q.moe_rmsnorm_mx(x, torch.ones(64), 1e-5, sum=x)
    with pytest.raises(ValueError, match="4-bit"):
        q.mx_experts(q.alloc_mx_rows((2, 32, 128), q.MOE_MX_E4M3, "cpu"))


def test_binding_checks_tables_of_the_product():
    w = q.MxExperts(mxdesc(E=4, N=128, K=128))
    a = q.alloc_mx_rows((8, 128), q.MOE_MX_E4M3, "cpu")
    seg = torch.zeros(5, dtype=torch.int32)
    pairs = torch.zeros(8, dtype=torch.int32)
    with pytest.raises(ValueError, match="seg_offsets"):
        q.moe_grouped_mxgemm(w, a, seg[:4], 8)
    with pytest.raises(ValueError, match="seg_offsets"):
        q.moe_grouped_mxgemm(w, a, seg.long(), 8)
    with pytest.raises(ValueError, match="gather_pair"):
        q.moe_grouped_mxgemm(w, a, seg, 16, gather_pair=pairs, k=2)
    with pytest.raises(ValueError, match="A must be"):
        q.moe_grouped_mxgemm(w, q.alloc_mx_rows((8, 256), q.MOE_MX_E4M3, "cpu"), seg, 8)
    with pytest.raises(ValueError, match="exactly"):
        q.moe_grouped_mxgemm(w, a, seg, 8, q.MOE_EPI_SWIGLU_E4M3, out=torch.zeros(8, 64))
    with pytest.raises(ValueError, match="epilogue"):
        q.moe_grouped_mxgemm(w, a, seg, 8, 9)
    with pytest.raises(ValueError, match="fit together"):
        q.moe_mx_layer_forward(torch.zeros(8, 128), torch.zeros(8, 4), 2, w, w)
