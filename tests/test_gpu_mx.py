"""GPU checks of the scored routing, the MX rows, the residual RMS norm, the
grouped MX product and the MX layer against float64 references
(oracle/mx_oracle.py).

Tolerances.  Ids, MX scale bytes and codes of given inputs are exact.  Weights
are float64 values rounded once to float32: 2^-24 relative, 2^-23 with the
order of float64 sums.  The norm's factor is float64, n takes a rounding of
the product (of fp32 rows) and its own, together below NORM = 2^-22.  One scaled matrix
instruction adds 64 products; it aligns them to the largest one and was
measured off by at most 2^-11 of it with an 8-bit operand, 2^-20 with two
4-bit ones; `bound` adds that over the K / 64 instructions, and half an fp32
ulp of the running sum (at most the sum of magnitudes) per instruction.
"""
import numpy as np
import pytest
import torch

import quantized_moe_expert_top_amd as q
from oracle import mx_oracle as mx

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
NORM = 2.0 ** -22
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
FMT = {"e4m3": q.MOE_MX_E4M3, "e2m1": q.MOE_MX_E2M1}
HALF_STEP = {mx.E4M3: (2.0 ** -4, 2.0 ** -10), mx.E2M1: (2.0 ** -2, 0.25)}  # relative; of the smallest step


def f64(t):
    return t.double().cpu().numpy()


def show(*a):
    print("[gpu]", *a, flush=True)


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


def decoded(rows):
    return mx.values(mx.unpack(rows.codes.cpu().numpy(), rows.fmt), rows.scales.cpu().numpy(), rows.fmt)


def close(got, ref, tol, what=""):
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off, first at {np.argwhere(bad)[0]}: " \
        f"{got[bad][0]} for {ref[bad][0]} (tolerance {np.broadcast_to(tol, ref.shape)[bad][0]})"


# ------------------------------------------------------------------- MX rows
def spiky(rng, rows, K, dt):
    """Normal values, a strong channel, a zero block, tiny and huge blocks, exact ties of both formats."""
    x = rng.standard_normal((rows, K)).astype(np.float32)
    x[:, K // 2] *= 30
    x[0, :32] = 0
    x[rows // 2, -32:] *= 2.0 ** (-20 if dt == "fp16" else -100)
    x[rows - 1, :32] = np.array([6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25] * 4, np.float32)
    if rows > 2:
        x[rows - 2, :32] = np.array([448, 440, 17, 19, 1.0625, 2.0 ** -10, 3 * 2.0 ** -10, -2.0 ** -10] * 4, np.float32)
    return dev(x, DT[dt])


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 96), (129, 2080), (64, 4096)])
def test_quantize_exact(fmt, dt, rows, K):
    x = spiky(np.random.default_rng(rows + K), rows, K, dt)
    show("quantize", fmt, dt, rows, K)
    r = q.moe_quantize_mx(x, FMT[fmt])
    codes, scales = mx.quantize(f64(x), FMT[fmt])
    assert np.array_equal(r.scales.cpu().numpy(), scales)
    got = mx.unpack(r.codes.cpu().numpy(), r.fmt)
    want = mx.values(codes, scales, r.fmt)
    assert np.array_equal(decoded(r), want)
    assert np.array_equal(got[want != 0], codes[want != 0])
    assert np.array_equal(f64(q.moe_dequantize_mx(r, torch.float32)), want)


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_quantize_extremes_and_not_finite(fmt):
    F = FMT[fmt]
    x = np.zeros((8, 32), np.float32)
    x[0, :] = 3.4028235e38
    x[1, :] = 1e-45          # the smallest subnormal
    x[2, 3] = np.inf
    x[3, 31] = np.nan
    x[4, 0] = -np.inf
    x[5, 7] = -2.0 ** -126
    x[6, :] = np.arange(32) - 16
    show("quantize extremes", fmt)
    r = q.moe_quantize_mx(dev(x), F)
    codes, scales = mx.quantize(x, F)
    assert np.array_equal(r.scales.cpu().numpy(), scales)
    assert (r.scales.cpu().numpy()[2:5] == 255).all() and (r.codes.cpu().numpy()[2:5] == 0).all()
    want = mx.values(codes, scales, F)
    np.testing.assert_array_equal(decoded(r), want)
    np.testing.assert_array_equal(f64(q.moe_dequantize_mx(r, torch.float32)), want.astype(np.float32).astype(np.float64))
    for dt in (torch.bfloat16, torch.float16):
        ref = torch.from_numpy(want.astype(np.float32)).to(dt).double().numpy()
        np.testing.assert_array_equal(f64(q.moe_dequantize_mx(r, dt)), ref)


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_dequantize_every_code_and_scale(fmt):
    """Every code byte under every scale byte, in fp32 (exact: the products are float32 values down to subnormals)."""
    F = FMT[fmt]
    per = 32 if fmt == "e4m3" else 16
    codes = np.tile(np.arange(256, dtype=np.uint8).reshape(-1, per), (256, 1))
    scales = np.repeat(np.arange(256, dtype=np.uint8), 256 // per)[:, None]
    show("dequantize all", fmt)
    got = f64(q.moe_dequantize_mx(q.MxRows(dev(codes), dev(scales), F), torch.float32))
    with np.errstate(over="ignore"):
        want = mx.values(mx.unpack(codes, F), scales, F).astype(np.float32).astype(np.float64)
    np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("shift", [0, -7, 40, -90])
def test_quantize_beside_every_border(fmt, shift):
    """fp32 values one step below, at and one step above every rounding border of the elements and of the scale."""
    F = FMT[fmt]
    t = mx.TABLE[F].astype(np.float32)
    mid = (t[1:] + t[:-1]) / 2  # exact in fp32
    v = np.concatenate([mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(1e9)),
                        np.nextafter(t[1:], np.float32(0)), np.nextafter(t[1:-1], np.float32(1e9)), t]).astype(np.float32)
    v = np.concatenate([v, -v])
    v = np.pad(v, (0, -len(v) % 31))
    x = np.concatenate([np.full((len(v) // 31, 1), t[-1]), v.reshape(-1, 31)], 1).astype(np.float32)  # scale 2^0 each
    top = np.full((2, 32), t[-1], np.float32)
    top[0, 5], top[1, 5] = np.nextafter(t[-1], np.float32(1e9)), np.nextafter(t[-1], np.float32(0))
    x = np.ldexp(np.concatenate([x, top]), shift).astype(np.float32)
    show("quantize borders", fmt, shift)
    r = q.moe_quantize_mx(dev(x), F)
    codes, scales = mx.quantize(x, F)
    assert np.array_equal(r.scales.cpu().numpy(), scales)
    assert np.array_equal(decoded(r), mx.values(codes, scales, F))


def test_offsets_past_32_bits():
    """Rows behind the 4 GiB and 2^31 element marks against the same rows on their own (bit for bit)."""
    def tail(t, n=96):
        return t[-n:].clone()
    g = torch.Generator(device=DEV).manual_seed(5)
    big = torch.empty(70001, 32768, device=DEV, dtype=torch.float16)   # 2.3e9 values
    big[-96:] = torch.randn(96, 32768, device=DEV, generator=g)
    big[:-96] = 1.0
    for fmt in (q.MOE_MX_E4M3, q.MOE_MX_E2M1):
        show("past 32 bits: quantise", fmt)
        r = q.moe_quantize_mx(big, fmt)
        one = q.moe_quantize_mx(tail(big), fmt)
        assert torch.equal(r.codes[-96:], one.codes) and torch.equal(r.scales[-96:], one.scales)
        show("past 32 bits: dequantise", fmt)
        back = q.moe_dequantize_mx(r)
        assert torch.equal(back[-96:], q.moe_dequantize_mx(one))
        assert (back[:3] == 1).all()
        del r, back
    x = big.view(-1, 8192)                                              # 280004 rows
    wn = torch.randn(8192, device=DEV, generator=g).half()
    show("past 32 bits: norm")
    a = q.moe_rmsnorm_mx(x, wn, 1e-5, residual=x, fmt=q.MOE_MX_E4M3, want_y=True)
    b = q.moe_rmsnorm_mx(tail(x), wn, 1e-5, residual=tail(x), fmt=q.MOE_MX_E4M3, want_y=True)
    assert torch.equal(a.sum[-96:], b.sum) and torch.equal(a.y[-96:], b.y) and torch.equal(a.rows.codes[-96:], b.rows.codes)
    del a, x, big
    show("past 32 bits: routing")
    logits = torch.zeros(2200000, 1024, device=DEV)
    logits[-96:] = torch.randn(96, 1024, device=DEV, generator=g)
    logits[:-96, 7] = 1.0
    ids, w = q.moe_route_scored(logits, 2, q.MOE_SCORE_SIGMOID)
    i1, w1 = q.moe_route_scored(tail(logits), 2, q.MOE_SCORE_SIGMOID)
    assert torch.equal(ids[-96:], i1) and torch.equal(w[-96:], w1) and (ids[:-96, 0] == 7).all()
    del logits
    # product: 4.6 GB of fp32 outputs, 2.1 GB of rows
    M, N, K = 140000, 8192, 16384
    codes = torch.full((M, K), 0x38, device=DEV, dtype=torch.uint8)    # 1.0
    codes[-96:] = q.moe_quantize_mx(torch.randn(96, K, device=DEV, generator=g)).codes
    A = q.MxRows(codes, torch.full((M, K // 32), 120, device=DEV, dtype=torch.uint8), q.MOE_MX_E4M3)
    wt = q.moe_mx_repack(q.mx_experts(q.moe_quantize_mx(torch.randn(1, N, K, device=DEV, generator=g), q.MOE_MX_E2M1)))
    seg = torch.tensor([0, M], device=DEV, dtype=torch.int32)
    for kernel in (q.MOE_KERNEL_TILE64, q.MOE_KERNEL_TILE128):
        show("past 32 bits: product", kernel)
        y = q.moe_grouped_mxgemm(wt, A, seg, M, q.MOE_EPI_NONE_F32, kernel=kernel)
        y1 = q.moe_grouped_mxgemm(wt, q.MxRows(tail(A.codes), tail(A.scales), A.fmt), torch.tensor([0, 96], device=DEV, dtype=torch.int32),
                                  96, q.MOE_EPI_NONE_F32, kernel=kernel)
        assert torch.equal(y[-96:], y1) and torch.equal(y[5], y[-97])


def test_quantize_leading_dims_out_and_empty():
    x = torch.randn(3, 5, 64, device=DEV)
    r = q.moe_quantize_mx(x, q.MOE_MX_E2M1)
    assert r.shape == (3, 5, 64) and q.moe_dequantize_mx(r).shape == (3, 5, 64)
    again = q.moe_quantize_mx(x, q.MOE_MX_E2M1, out=q.alloc_mx_rows((3, 5, 64), q.MOE_MX_E2M1, DEV))
    assert torch.equal(r.codes, again.codes) and torch.equal(r.scales, again.scales)
    assert q.moe_quantize_mx(x[:0]).codes.shape == (0, 5, 64)
    with pytest.raises(ValueError):
        q.moe_quantize_mx(x, q.MOE_MX_E4M3, out=r)
    with pytest.raises(ValueError, match="contiguous"):
        q.moe_quantize_mx(x.transpose(0, 1))
    with pytest.raises(q.MoeError):
        q.moe_quantize_mx(torch.zeros(4 * 64 + 2, device=DEV)[2:].view(4, 64))  # 8-byte aligned


# -------------------------------------------------------------------- the norm
def check_mx_near(got, ref, tol, F, what):
    """MX values `got` of numbers within `tol` of `ref`: half a step of the element (of the next larger scale where
    the block's largest is at a border)."""
    p = np.repeat(mx.scale_exponent(np.abs(ref).reshape(*ref.shape[:-1], -1, 32).max(-1), F), 32, -1)
    rel, least = HALF_STEP[F]
    close(got, ref, np.maximum(rel * np.abs(ref), least * np.exp2(p + 1.0)) + 1.5 * tol, what)


@pytest.mark.parametrize("rows,H", [(1, 32), (7, 96), (5, 512), (3, 544), (33, 2048), (2, 4096), (3, 8160), (2, 16384),
                                    (513, 2080), (520, 4096), (515, 5120), (514, 8192)])
@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_rmsnorm(rows, H, dt, fmt):
    rng = np.random.default_rng(H + rows)
    x, r = (dev(rng.standard_normal((rows, H)).astype(np.float32) * s, DT[dt]) for s in (1.0, 3.0))
    w = dev((1 + 0.2 * rng.standard_normal(H)).astype(np.float32), DT[dt])
    eps = 1e-5
    show("rmsnorm", rows, H, dt, fmt)
    o = q.moe_rmsnorm_mx(x, w, eps, residual=r, fmt=FMT[fmt], want_y=True)
    v = f64((x.double() + r.double()).to(DT[dt]))
    assert np.array_equal(f64(o.sum), v)
    n = mx.rmsnorm(v, f64(w), eps)
    close(f64(o.y), n, (torch.finfo(DT[dt]).eps / 2 + NORM) * np.abs(n) + 1e-7 * (dt == "fp16"), "y")
    check_mx_near(decoded(o.rows), n, NORM * np.abs(n), FMT[fmt], "rows")
    # n is known to about 2^-46 and rounded to odd before it is quantised: the MX rows are exactly those of n
    assert np.array_equal(decoded(o.rows), mx.values(*mx.quantize(n, FMT[fmt]), FMT[fmt]))


def test_rmsnorm_outputs_in_place_and_zero_rows():
    x, r = torch.randn(9, 256, device=DEV).bfloat16(), torch.randn(9, 256, device=DEV).bfloat16()
    x[4], r[4] = 0, 0
    w = torch.randn(256, device=DEV).bfloat16()
    full = q.moe_rmsnorm_mx(x, w, 1e-6, residual=r, want_y=True)
    only_y = q.moe_rmsnorm_mx(x, w, 1e-6, residual=r, fmt=None, want_y=True)
    assert only_y.rows is None and torch.equal(only_y.y, full.y)
    plain = q.moe_rmsnorm_mx(full.sum, w, 1e-6)
    assert plain.sum is None and plain.y is None
    assert torch.equal(plain.rows.codes, full.rows.codes) and torch.equal(plain.rows.scales, full.rows.scales)
    assert (full.y[4] == 0).all() and (full.rows.codes[4] == 0).all()
    r2, x2 = r.clone(), x.clone()
    o = q.moe_rmsnorm_mx(x2, w, 1e-6, residual=r2, sum=r2, y=x2)  # the residual stream updated, the norm over x
    assert torch.equal(r2, full.sum) and torch.equal(x2, full.y) and torch.equal(o.rows.codes, full.rows.codes)
    zero = q.moe_rmsnorm_mx(x[4:5], w, 0.0, want_y=True)  # 0 / 0: not a number, as the formula says
    assert torch.isnan(zero.y).all() and (zero.rows.scales == 255).all()
    assert q.moe_rmsnorm_mx(x[:0], w, 1e-6).rows.codes.shape == (0, 256)
    x[2, 7] = float("nan")
    o = q.moe_rmsnorm_mx(x, w, 1e-6, residual=r, want_y=True)
    keep = [i for i in range(9) if i != 2]
    assert torch.isnan(o.y[2]).all() and (o.rows.scales[2] == 255).all() and torch.equal(o.y[keep], full.y[keep])


# --------------------------------------------------------------------- routing
def check_route(logits, k, **kw):
    bias = kw.pop("bias", None)
    score = kw.pop("sigmoid", False)
    args = dict(n_group=kw.get("n_group", 1), topk_group=kw.get("topk_group", 1), group_top=kw.get("group_top", 1),
                renormalize=kw.get("renorm", True), scale=kw.get("scale", 1.0))
    show("route", logits.shape, k, args, "bias" if bias is not None else "", "sigmoid" if score else "softmax")
    ids, w = q.moe_route_scored(dev(logits), k, score=q.MOE_SCORE_SIGMOID if score else q.MOE_SCORE_SOFTMAX,
                                bias=None if bias is None else dev(bias), **args)
    ref_ids, ref_w = mx.route_scored(logits, k, sigmoid=score, bias=bias, **kw)
    assert np.array_equal(ids.cpu().numpy(), ref_ids)
    np.testing.assert_allclose(f64(w), ref_w, rtol=2.0 ** -23, atol=1e-45)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("T,E,k,G,tg,gt", [(1, 1, 1, 1, 1, 1), (1, 64, 8, 1, 1, 1), (37, 60, 4, 1, 1, 2), (9, 64, 64, 1, 1, 1),
                                           (33, 64, 6, 8, 3, 1), (5, 128, 8, 1, 1, 1), (21, 130, 7, 5, 2, 2),
                                           (50, 256, 8, 8, 4, 2), (3, 1000, 16, 40, 20, 1), (4, 1024, 33, 64, 64, 2),
                                           (6, 512, 5, 1, 1, 1), (2, 96, 40, 48, 24, 2)])
def test_route_scored(sigmoid, with_bias, T, E, k, G, tg, gt):
    rng = np.random.default_rng(T * E + k)
    logits = (2 * rng.standard_normal((T, E))).astype(np.float32)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32) if with_bias else None
    check_route(logits, k, sigmoid=sigmoid, bias=bias, n_group=G, topk_group=tg, group_top=gt)
    check_route(logits, k, sigmoid=sigmoid, bias=bias, n_group=G, topk_group=tg, group_top=gt, renorm=False, scale=2.5)


@pytest.mark.parametrize("E", [8, 64, 200, 1024])
def test_route_scored_ties(E):
    rng = np.random.default_rng(E)
    logits = rng.integers(-1, 2, size=(40, E)).astype(np.float32)
    logits[0] = 0
    for sigmoid in (False, True):
        check_route(logits, min(E, 9), sigmoid=sigmoid)
        check_route(logits, min(E, 5), sigmoid=sigmoid, n_group=4, topk_group=2)
    logits[1:20] *= 100  # saturated scores: equal in float64, lower index first
    check_route(logits, min(E, 9), sigmoid=True, renorm=False)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E,G,gt", [(48, 1, 1), (64, 4, 1), (64, 4, 2), (256, 8, 2), (1000, 10, 1)])
def test_route_scored_near_ties(sigmoid, E, G, gt):
    """Scores closer than fp32 tells apart: single fp32 steps of equal logits, differences of 1e-6, saturated scores."""
    rng = np.random.default_rng(E + G + gt)
    logits = (1.5 + 1e-6 * rng.standard_normal((24, E))).astype(np.float32)
    if gt == 1:
        logits[:8] = np.float32(1.5) + rng.integers(0, 6, (8, E)).astype(np.float32) * np.float32(2.0 ** -23)
        logits[8:12] += 21  # sigmoid: 1 - 2e-10, steps of 1e-16
    bias = (1e-6 * rng.standard_normal(E)).astype(np.float32)
    for b in (None, bias):
        check_route(logits, 7, sigmoid=sigmoid, bias=b, n_group=G, topk_group=max(1, G // 2), group_top=gt)
    check_route(logits, 7, sigmoid=sigmoid, n_group=G, topk_group=max(1, G // 2), group_top=gt, renorm=False)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E,G", [(16, 1), (16, 4), (96, 8), (256, 16)])
def test_route_scored_barred_experts(sigmoid, E, G):
    """-inf and NaN logits and biases bar experts; rows with too few, one and no expert left; +inf counts as FLT_MAX."""
    rng = np.random.default_rng(E + G)
    logits = rng.standard_normal((12, E)).astype(np.float32)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    bias[3], bias[7] = -np.inf, np.nan
    logits[0] = -np.inf
    logits[1] = np.nan
    logits[2, 1:] = -np.inf
    logits[3, ::2] = -np.inf
    logits[4, 5] = np.inf
    logits[5] = -3.4028235e38
    logits[6, : E // 2] = np.nan
    for b in (None, bias):
        check_route(logits, 6, sigmoid=sigmoid, bias=b, n_group=G, topk_group=max(1, G // 2), group_top=2)


def test_route_scored_empty_and_buffers():
    ids, w = q.moe_route_scored(torch.zeros(0, 8, device=DEV), 2)
    assert ids.shape == (0, 2) and w.shape == (0, 2)
    x = torch.randn(5, 16, device=DEV)
    ids, w = torch.empty(5, 3, dtype=torch.int32, device=DEV), torch.empty(5, 3, device=DEV)
    got = q.moe_route_scored(x, 3, ids=ids, w=w)
    assert got[0] is ids and torch.equal(ids, q.moe_route_scored(x, 3)[0])
    old_ids, old_w = q.moe_route_topk(x, 3)  # softmax scores renormalised over the chosen: the expert gate
    assert torch.equal(ids, old_ids) and torch.allclose(w, old_w, rtol=2.0 ** -22, atol=0)
    with pytest.raises(ValueError):
        q.moe_route_scored(x, 3, ids=ids[:, :2])
    with pytest.raises(q.MoeError):
        q.moe_route_scored(x, 3, n_group=3)


# ----------------------------------------------------------------- the product
class Product:
    """One grouped product: MX experts, MX rows and segments, with float64 values of both."""

    def __init__(self, seed, E, N, K, act, counts, k=1, gather=True, lead=0):
        rng = np.random.default_rng(seed)
        self.E, self.N, self.K, self.k = E, N, K, k
        w = rng.standard_normal((E, N, K)) * np.exp2(rng.integers(-3, 4, (E, N, 1)))
        self.canon = q.moe_quantize_mx(dev(w.astype(np.float32)), q.MOE_MX_E2M1)
        self.tiled = q.moe_mx_repack(q.mx_experts(self.canon))
        self.wv = decoded(self.canon)
        M = int(sum(counts))
        self.lead, self.M = lead, M
        rows = M if not gather else max(1, -(-(M + lead) // k))
        self.A = q.moe_quantize_mx(dev((rng.standard_normal((rows + lead, K)) * np.exp2(rng.integers(-2, 3, (rows + lead, 1)))
                                        ).astype(np.float32)), FMT[act])
        self.av = decoded(self.A)
        self.seg = np.concatenate([[lead], lead + np.cumsum(counts)]).astype(np.int32)
        self.pairs = rng.integers(0, (rows + lead) * k, M + lead).astype(np.int32) if gather else None
        self.F = FMT[act]

    def reference(self):
        src = self.pairs // self.k if self.pairs is not None else np.arange(self.M + self.lead)
        a = self.av[src]
        y = np.zeros((self.M + self.lead, self.N))
        tol = np.zeros_like(y)
        eps = 2.0 ** (-11 if self.F == mx.E4M3 else -20)
        top = lambda v: np.abs(v).reshape(*v.shape[:-1], v.shape[-1] // 64, 64).max(-1)  # noqa: E731
        for e in range(self.E):
            s = slice(self.seg[e], self.seg[e + 1])
            y[s] = a[s] @ self.wv[e].T
            tol[s] = eps * (top(a[s]) @ top(self.wv[e]).T) + self.K / 64 * 2.0 ** -24 * (np.abs(a[s]) @ np.abs(self.wv[e]).T)
        return y, tol

    def run(self, epi, kernel, out=None):
        return q.moe_grouped_mxgemm(self.tiled, self.A, dev(self.seg), self.M + self.lead, epi,
                                    gather_pair=None if self.pairs is None else dev(self.pairs), k=self.k, out=out,
                                    kernel=kernel)


KERNELS = [q.MOE_KERNEL_AUTO, q.MOE_KERNEL_SMALL, q.MOE_KERNEL_TILE64, q.MOE_KERNEL_TILE128]
OUT_EPS = {q.MOE_EPI_NONE: 2.0 ** -8, q.MOE_EPI_NONE_F32: 2.0 ** -24, q.MOE_EPI_NONE_F16: 2.0 ** -11,
           q.MOE_EPI_SWIGLU: 2.0 ** -8}


def swiglu(y, tol):
    g, u = np.split(y, 2, -1)
    dg, du = np.split(tol, 2, -1)
    with np.errstate(over="ignore"):
        sg = g / (1 + np.exp(-g))
    h = sg * u
    # |silu'| <= 1.1; exp, reciprocal and three products in fp32: below 2^-20 relative
    return h, 1.1 * np.abs(u) * dg + np.abs(sg) * du + 1.1 * dg * du + 2.0 ** -20 * np.abs(h)


def check_product(p, epi, kernel, what):
    show("product", what, "epi", epi, "kernel", kernel)
    y, tol = p.reference()
    rows = slice(p.lead, p.lead + p.M)
    if epi in (q.MOE_EPI_SWIGLU_E4M3, q.MOE_EPI_SWIGLU_E2M1):
        F = mx.E4M3 if epi == q.MOE_EPI_SWIGLU_E4M3 else mx.E2M1
        h, tol = swiglu(y, tol)
        check_mx_near(decoded(p.run(epi, kernel))[rows], h[rows], tol[rows], F, what)
        return
    if epi == q.MOE_EPI_SWIGLU:
        y, tol = swiglu(y, tol)
    ref = y[rows]
    got = f64(p.run(epi, kernel))[rows]
    close(got, ref, OUT_EPS[epi] * np.abs(ref) + tol[rows] * (1 + 2.0 ** -8) + 2.0 ** -24, what)
    if ref.size:
        assert np.linalg.norm(got - ref) <= 5e-3 * np.linalg.norm(ref), what


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("act", ["e4m3", "e2m1"])
@pytest.mark.parametrize("epi", [q.MOE_EPI_NONE, q.MOE_EPI_SWIGLU, q.MOE_EPI_NONE_F32, q.MOE_EPI_NONE_F16,
                                 q.MOE_EPI_SWIGLU_E4M3, q.MOE_EPI_SWIGLU_E2M1])
def test_product_every_epilogue(kernel, act, epi):
    """Segments of no, one, a few and more than two tiles of rows, through a gather."""
    p = Product(5, 5, 192, 384, act, [0, 1, 37, 300, 0], k=3)
    check_product(p, epi, kernel, f"{act} 192x384")


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("act", ["e4m3", "e2m1"])
@pytest.mark.parametrize("E,N,K,counts", [(1, 32, 128, [1]), (1, 64, 128, [129]), (3, 96, 256, [64, 65, 63]),
                                          (2, 544, 640, [128, 17]), (4, 64, 2048, [5, 0, 0, 140]),
                                          (2, 320, 1152, [31, 257])])
def test_product_sizes(kernel, act, E, N, K, counts):
    p = Product(N + K, E, N, K, act, counts, gather=False)
    check_product(p, q.MOE_EPI_NONE_F16 if N % 64 else q.MOE_EPI_SWIGLU_E4M3, kernel, f"{act} {N}x{K} {counts}")
    check_product(p, q.MOE_EPI_NONE, kernel, f"{act} {N}x{K} {counts}")


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("act", ["e4m3", "e2m1"])
@pytest.mark.parametrize("epi", [q.MOE_EPI_NONE_F32, q.MOE_EPI_SWIGLU_E4M3])
@pytest.mark.parametrize("K", [128, 640])
def test_product_last_rows(kernel, act, epi, K):
    """Segments whose last tile holds up to a quarter, a half, three quarters and all of its rows."""
    p = Product(K + 7, 10, 64, K, act, [32, 33, 64, 65, 96, 97, 160, 161, 224, 225], k=2)
    check_product(p, epi, kernel, f"{act} 64x{K}")


SPLIT = [("e4m3", q.MOE_KERNEL_TILE64), ("e2m1", q.MOE_KERNEL_TILE64_SPLIT_K)]


@pytest.mark.parametrize("act,kernel", SPLIT)
@pytest.mark.parametrize("epi", [q.MOE_EPI_NONE, q.MOE_EPI_SWIGLU, q.MOE_EPI_NONE_F32, q.MOE_EPI_NONE_F16,
                                 q.MOE_EPI_SWIGLU_E4M3, q.MOE_EPI_SWIGLU_E2M1])
@pytest.mark.parametrize("K", [384, 512, 640, 2176, 2304, 2560, 4224])
def test_product_long_k(act, kernel, epi, K):
    """64-row tiles (of e2m1 rows with K split over two groups of wavefronts): even, odd and half chunks of 256."""
    p = Product(K, 3, 320, K, act, [1, 0, 133], k=3)
    check_product(p, epi, kernel, f"{act} 320x{K}")


@pytest.mark.parametrize("act,kernel", SPLIT)
def test_product_long_k_other_rows_and_not_a_number(act, kernel):
    p = Product(21, 2, 64, 2304, act, [70, 30], gather=False, lead=5)
    for row, block in ((8, 3), (70, 71)):
        p.A.scales[row, block] = 255
    out = torch.full((p.lead + p.M + 4, 64), 7.0, device=DEV)
    p.A = q.MxRows(torch.cat([p.A.codes] * 2), torch.cat([p.A.scales] * 2), p.A.fmt)
    q.moe_grouped_mxgemm(p.tiled, p.A, dev(p.seg), out.shape[0], q.MOE_EPI_NONE_F32, out=out, kernel=kernel)
    assert (out[:5] == 7).all() and (out[-4:] == 7).all()
    nan = torch.isnan(out).all(-1)
    assert nan[8] and nan[70] and int(nan.sum()) == 2 and int(torch.isnan(out).any(-1).sum()) == 2
    again = q.moe_grouped_mxgemm(p.tiled, p.A, dev(p.seg), out.shape[0], q.MOE_EPI_NONE_F32, out=torch.full_like(out, 7.0),
                                 kernel=kernel)
    assert torch.equal(out.view(torch.int32), again.view(torch.int32))


@pytest.mark.parametrize("kernel", KERNELS)
def test_product_leaves_other_rows(kernel):
    """A slice of a longer segment table: rows before it, between nothing and behind it stay as they were; the same
    call gives the same bits again."""
    p = Product(9, 3, 128, 256, "e4m3", [40, 0, 90], k=2, lead=11)
    total = p.lead + p.M + 8
    p.pairs = np.concatenate([p.pairs, np.zeros(8, np.int32)])
    out = torch.full((total, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    call = lambda o: q.moe_grouped_mxgemm(p.tiled, p.A, dev(p.seg), total, q.MOE_EPI_NONE, gather_pair=dev(p.pairs),  # noqa: E731
                                          k=2, out=o, kernel=kernel)
    p.A = q.MxRows(torch.cat([p.A.codes] * 2), torch.cat([p.A.scales] * 2), p.A.fmt)  # A_rows * k >= M_total
    call(out)
    assert (out[: p.lead] == 7).all() and (out[p.lead + p.M:] == 7).all()
    assert not (out[p.lead: p.lead + p.M] == 7).all(-1).any()
    assert torch.equal(out, call(torch.full_like(out, 7.0)))
    h = q.alloc_mx_rows((total, 64), q.MOE_MX_E4M3, DEV)
    h.codes.fill_(99), h.scales.fill_(98)
    q.moe_grouped_mxgemm(p.tiled, p.A, dev(p.seg), total, q.MOE_EPI_SWIGLU_E4M3, gather_pair=dev(p.pairs), k=2, out=h,
                         kernel=kernel)
    for t, v in ((h.codes, 99), (h.scales, 98)):
        assert (t[: p.lead] == v).all() and (t[p.lead + p.M:] == v).all()


@pytest.mark.parametrize("kernel", KERNELS)
def test_product_not_a_number_stays_in_its_row(kernel):
    p = Product(11, 2, 64, 128, "e4m3", [70, 30], gather=False)
    p.A.scales[13, 2] = 255
    out = p.run(q.MOE_EPI_NONE_F32, kernel)
    assert torch.isnan(out[13]).all() and not torch.isnan(out[:13]).any() and not torch.isnan(out[14:]).any()
    h = p.run(q.MOE_EPI_SWIGLU_E4M3, kernel)
    assert (h.scales[13] == 255).all() and (h.scales[14:] != 255).all()


def test_product_no_rows_and_refusals():
    p = Product(3, 2, 64, 128, "e4m3", [0, 0], gather=False)
    assert q.moe_grouped_mxgemm(p.tiled, p.A, dev(p.seg), 0).shape == (0, 64)
    out = torch.full((4, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    a = q.alloc_mx_rows((4, 128), q.MOE_MX_E4M3, DEV)
    q.moe_grouped_mxgemm(p.tiled, a, dev(p.seg), 4, out=out)  # every segment empty
    assert (out == 3).all()
    with pytest.raises(q.MoeError):
        q.moe_grouped_mxgemm(q.mx_experts(p.canon), a, dev(p.seg), 4)  # canonical weights
    with pytest.raises(q.MoeError):
        q.moe_grouped_mxgemm(p.tiled, a, dev(p.seg), 5)  # more rows than A holds
    with pytest.raises(ValueError):
        q.moe_grouped_mxgemm(p.tiled, a, dev(p.seg), 4, out=out.half())


# ------------------------------------------------------------------- the layer
def layer_reference(av, logits, k, gu, dn, h_fmt, routing):
    """float64 layer on decoded values: ids, weights, output, and a tolerance that follows the product's bound and one
    element step of the SwiGLU activations at rounding borders."""
    ids, w = mx.route_scored(logits, k, **routing)
    T, H = av.shape
    out, tol = np.zeros((T, H)), np.zeros((T, H))
    rel, least = HALF_STEP[h_fmt]
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            if e < 0:
                continue
            y = gu[e] @ av[t]
            g, u = np.split(y, 2)
            h = g / (1 + np.exp(-g)) * u
            hq = mx.values(*mx.quantize(h, h_fmt), h_fmt)
            yv = dn[e] @ hq
            out[t] += w[t, j] * yv
            tol[t] += np.abs(w[t, j]) * (2.0 ** -11 * np.abs(yv))
    return ids, w, out, tol


@pytest.mark.parametrize("T", [1, 5, 64])
@pytest.mark.parametrize("act,h_fmt", [("e4m3", "e4m3"), ("e2m1", "e4m3"), ("e4m3", "e2m1")])
def test_layer(T, act, h_fmt):
    """norm -> scored routing -> grouping -> products -> combine as they would be used, against float64.  The bar
    is the framework's layer bar (relative L2 5e-3) with two 2^-8 roundings (bf16 output, fp16 expert outputs)
    inside it; activations on the other side of a rounding border move single elements of one expert's h."""
    E, H, I, k = 8, 256, 384, 3
    rng = np.random.default_rng(T)
    g = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
    gu = q.moe_quantize_mx(dev(g(E, 2 * I, H) / 16), q.MOE_MX_E2M1)
    dn = q.moe_quantize_mx(dev(g(E, H, I) / 20), q.MOE_MX_E2M1)
    x, res = dev(g(T, H), torch.bfloat16), dev(2 * g(T, H), torch.bfloat16)
    wn = dev(1 + 0.1 * g(H), torch.bfloat16)
    logits = g(T, E)
    bias = 0.05 * g(E)
    if T > 4:
        logits[2] = -np.inf      # a padded token: no expert
        logits[3, 1:] = np.nan   # one expert only
    show("layer", T, act, h_fmt)
    rows = q.moe_rmsnorm_mx(x, wn, 1e-5, residual=res, fmt=FMT[act]).rows
    buf = q.alloc_mx_layer(T, E, k, H, I, DEV, act=FMT[act], h_fmt=FMT[h_fmt])
    q.moe_mx_layer_forward(rows, dev(logits), k, q.moe_mx_repack(q.mx_experts(gu)), q.moe_mx_repack(q.mx_experts(dn)),
                           routing=q.ScoredRouting(score=q.MOE_SCORE_SIGMOID, bias=dev(bias), scale=1.5), buf=buf)
    ids, w, out, _ = layer_reference(decoded(rows), logits, k, decoded(gu), decoded(dn), FMT[h_fmt],
                                     dict(sigmoid=True, bias=bias, scale=1.5))
    assert np.array_equal(buf.ids.cpu().numpy(), ids)
    np.testing.assert_allclose(f64(buf.w), w, rtol=2.0 ** -23, atol=0)
    got = f64(buf.out)
    assert np.linalg.norm(got - out) <= 5e-3 * np.linalg.norm(out)
    if T > 4:
        assert (got[2] == 0).all() and (ids[2] == -1).all()


def test_layer_quantises_bf16_input_and_checks_sizes():
    E, H, I, k, T = 4, 128, 128, 2, 9
    gu = q.moe_mx_repack(q.mx_experts(q.moe_quantize_mx(torch.randn(E, 2 * I, H, device=DEV), q.MOE_MX_E2M1)))
    dn = q.moe_mx_repack(q.mx_experts(q.moe_quantize_mx(torch.randn(E, H, I, device=DEV), q.MOE_MX_E2M1)))
    x, logits = torch.randn(T, H, device=DEV).bfloat16(), torch.randn(T, E, device=DEV)
    a = q.moe_mx_layer_forward(x, logits, k, gu, dn)
    b = q.moe_mx_layer_forward(q.moe_quantize_mx(x), logits, k, gu, dn, buf=q.alloc_mx_layer(T, E, k, H, I, DEV))
    assert torch.equal(a.out, b.out) and a.out.abs().sum() > 0
    with pytest.raises(ValueError, match="buffers"):
        q.moe_mx_layer_forward(x[:5].contiguous(), logits[:5].contiguous(), k, gu, dn, buf=a)
    assert q.moe_mx_layer_forward(x[:0], logits[:0], k, gu, dn).out.shape == (0, H)


@pytest.mark.parametrize("T,E,k,given", [(1, 4, 1, False), (16, 256, 8, False), (16, 64, 6, True), (17, 64, 6, False),
                                         (9, 300, 5, False), (3, 100, 33, False), (700, 40, 8, True), (1200, 130, 4, False),
                                         (300, 1000, 2, False), (8192, 12, 2, False), (8200, 5, 1, False),
                                         (17409, 63, 1, False), (9000, 128, 2, True), (2000, 520, 2, False),
                                         (3000, 1000, 2, False), (70000, 63, 1, False), (33000, 200, 1, False)])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_layer_call_equals_its_parts(T, E, k, given, dt):
    """The layer's one call (fused starts for few tokens, separate launches for many) against routing, grouping,
    quantisation, products and combine called one by one: every buffer bit for bit."""
    H, I = 128, 128
    g = torch.Generator(device=DEV).manual_seed(T + E)
    r = lambda *s: torch.randn(*s, device=DEV, generator=g)  # noqa: E731
    gu = q.moe_mx_repack(q.mx_experts(q.moe_quantize_mx(r(E, 2 * I, H), q.MOE_MX_E2M1)))
    dn = q.moe_mx_repack(q.mx_experts(q.moe_quantize_mx(r(E, H, I), q.MOE_MX_E2M1)))
    x, logits, bias = r(T, H).to(DT[dt]), r(T, E), 0.1 * r(E)
    if T > 2:
        logits[1] = -float("inf")
        logits[2, 1:] = float("nan")
    show("layer parts", T, E, k, given, dt)
    for routing in (q.ScoredRouting(), q.ScoredRouting(score=q.MOE_SCORE_SIGMOID, bias=bias, renormalize=False, scale=2.5),
                    q.ScoredRouting(bias=bias, n_group=4 if E % 4 == 0 else 1, topk_group=2 if E % 4 == 0 else 1, group_top=2)):
        rows = q.moe_quantize_mx(x, q.MOE_MX_E2M1)
        buf = q.alloc_mx_layer(T, E, k, H, I, DEV, act=q.MOE_MX_E2M1)
        for t in (buf.out, buf.y_perm, buf.w):
            t.fill_(7)
        q.moe_mx_layer_forward(rows if given else x, logits, k, gu, dn, routing=routing, buf=buf)
        ids, w = q.moe_route_scored(logits, k, routing.score, routing.bias, routing.n_group, routing.topk_group,
                                    routing.group_top, routing.renormalize, routing.scale)
        p = q.moe_permute(ids, E)
        h = q.moe_grouped_mxgemm(gu, rows, p.seg_offsets, T * k, q.MOE_EPI_SWIGLU_E4M3, gather_pair=p.sorted_pair, k=k)
        y = q.moe_grouped_mxgemm(dn, h, p.seg_offsets, T * k, q.MOE_EPI_NONE_F16)
        out = q.moe_unpermute_combine(y, p.pair_pos, w, T, k, n_valid=p.seg_offsets[-1:])
        n = int(p.seg_offsets[-1])
        assert torch.equal(buf.ids, ids) and torch.equal(buf.w, w) and torch.equal(buf.out, out)
        for a, b in ((buf.perm.counts, p.counts), (buf.perm.seg_offsets, p.seg_offsets),
                     (buf.perm.sorted_pair, p.sorted_pair), (buf.perm.pair_pos, p.pair_pos),
                     (buf.h.codes[:n], h.codes[:n]), (buf.h.scales[:n], h.scales[:n]), (buf.y_perm[:n], y[:n])):
            assert torch.equal(a, b)
        if not given:
            assert torch.equal(buf.x.codes, rows.codes) and torch.equal(buf.x.scales, rows.scales)


@pytest.mark.parametrize("y_dtype,epi", [(torch.float32, q.MOE_EPI_NONE_F32), (torch.bfloat16, q.MOE_EPI_NONE),
                                         (torch.float16, q.MOE_EPI_NONE_F16)])
@pytest.mark.parametrize("kernel", KERNELS + [q.MOE_KERNEL_TILE64_SPLIT_K])
@pytest.mark.parametrize("h_fmt", [q.MOE_MX_E4M3, q.MOE_MX_E2M1])
def test_layer_choices(y_dtype, epi, kernel, h_fmt):
    """Expert outputs of every type, hidden rows of either format, every kernel: the parts' bits."""
    E, H, I, k, T = 6, 384, 512, 3, 70
    g = torch.Generator(device=DEV).manual_seed(3)
    r = lambda *s: torch.randn(*s, device=DEV, generator=g)  # noqa: E731
    gu = q.moe_mx_repack(q.mx_experts(q.moe_quantize_mx(r(E, 2 * I, H), q.MOE_MX_E2M1)))
    dn = q.moe_mx_repack(q.mx_experts(q.moe_quantize_mx(r(E, H, I) / 20, q.MOE_MX_E2M1)))
    x, logits = r(T, H).half(), r(T, E)
    show("layer choices", y_dtype, kernel, h_fmt)
    act = q.MOE_MX_E2M1 if kernel == q.MOE_KERNEL_TILE64_SPLIT_K else q.MOE_MX_E4M3
    buf = q.alloc_mx_layer(T, E, k, H, I, DEV, act=act, h_fmt=h_fmt, y_dtype=y_dtype)
    if kernel == q.MOE_KERNEL_TILE64_SPLIT_K and h_fmt == q.MOE_MX_E4M3:
        with pytest.raises(RuntimeError, match="e2m1"):
            q.moe_mx_layer_forward(x, logits, k, gu, dn, buf=buf, kernel=kernel)
        return
    q.moe_mx_layer_forward(x, logits, k, gu, dn, buf=buf, kernel=kernel)
    ids, w = q.moe_route_scored(logits, k)
    p = q.moe_permute(ids, E)
    h = q.moe_grouped_mxgemm(gu, q.moe_quantize_mx(x, act), p.seg_offsets, T * k,
                             q.MOE_EPI_SWIGLU_E4M3 if h_fmt == q.MOE_MX_E4M3 else q.MOE_EPI_SWIGLU_E2M1,
                             gather_pair=p.sorted_pair, k=k, kernel=kernel)
    y = q.moe_grouped_mxgemm(dn, h, p.seg_offsets, T * k, epi, kernel=kernel)
    assert y.dtype == y_dtype and torch.equal(buf.y_perm, y) and torch.equal(buf.h.codes, h.codes)
    assert torch.equal(buf.out, q.moe_unpermute_combine(y, p.pair_pos, w, T, k, n_valid=p.seg_offsets[-1:]))


def test_layers_at_once():
    """Two layers on two streams, and the same layer from two threads with buffers of their own: the bits of calls
    one after another."""
    import threading
    E, H, I, k, T = 8, 256, 384, 2, 300
    g = torch.Generator(device=DEV).manual_seed(8)
    r = lambda *s: torch.randn(*s, device=DEV, generator=g)  # noqa: E731
    gu = q.moe_mx_repack(q.mx_experts(q.moe_quantize_mx(r(E, 2 * I, H), q.MOE_MX_E2M1)))
    dn = q.moe_mx_repack(q.mx_experts(q.moe_quantize_mx(r(E, H, I), q.MOE_MX_E2M1)))
    x, logits = [r(T, H).bfloat16() for _ in range(2)], [r(T, E) for _ in range(2)]
    want = [q.moe_mx_layer_forward(x[i], logits[i], k, gu, dn).out for i in range(2)]
    bufs = [q.alloc_mx_layer(T, E, k, H, I, DEV) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()

    def work(i):
        for _ in range(20):
            q.moe_mx_layer_forward(x[i], logits[i], k, gu, dn, buf=bufs[i], stream=streams[i])
    for how in ("streams", "threads"):
        for b in bufs:
            b.out.zero_()
        torch.cuda.synchronize()
        if how == "streams":
            work(0), work(1)
        else:
            ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
            [t.start() for t in ts], [t.join() for t in ts]
        torch.cuda.synchronize()
        assert torch.equal(bufs[0].out, want[0]) and torch.equal(bufs[1].out, want[1]), how


@pytest.mark.parametrize("T", [8, 24, 3000])
def test_layer_captured_and_on_other_streams(T):
    """The run of operators captured into a graph, replayed on new inputs with eager work between the replays, and
    issued on a side stream: the eager bits each time."""
    E, H, I, k = 8, 256, 256, 2
    gu = q.moe_mx_repack(q.mx_experts(q.moe_quantize_mx(torch.randn(E, 2 * I, H, device=DEV), q.MOE_MX_E2M1)))
    dn = q.moe_mx_repack(q.mx_experts(q.moe_quantize_mx(torch.randn(E, H, I, device=DEV), q.MOE_MX_E2M1)))
    wn = torch.ones(H, device=DEV).bfloat16()
    x, res = torch.randn(T, H, device=DEV).bfloat16(), torch.randn(T, H, device=DEV).bfloat16()
    logits = torch.randn(T, E, device=DEV)
    buf = q.alloc_mx_layer(T, E, k, H, I, DEV)
    s_out, rows = torch.empty_like(x), q.alloc_mx_rows((T, H), q.MOE_MX_E4M3, DEV)

    def step(stream=None, buf=buf, rows=rows, s_out=s_out):
        q.moe_rmsnorm_mx(x, wn, 1e-5, residual=res, sum=s_out, out=rows, stream=stream)
        return q.moe_mx_layer_forward(rows, logits, k, gu, dn, buf=buf, stream=stream)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    other = (q.alloc_mx_layer(T, E, k, H, I, DEV), q.alloc_mx_rows((T, H), q.MOE_MX_E4M3, DEV), torch.empty_like(x))
    for i in range(4):
        x.copy_(torch.randn(T, H, device=DEV))
        logits.copy_(torch.randn(T, E, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        want = step(None, *other)
        torch.cuda.synchronize()
        assert torch.equal(buf.out, want.out) and torch.equal(buf.ids, want.ids) and torch.equal(s_out, other[2])
        side.wait_stream(torch.cuda.current_stream())
        on_side = q.moe_mx_layer_forward(other[1], logits, k, gu, dn, stream=side)  # allocates on the side stream
        side.synchronize()
        assert torch.equal(on_side.out, want.out)
