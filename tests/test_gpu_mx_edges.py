"""GPU checks of the MX operators at the ends of their ranges, against the
float64 references (oracle/mx_oracle.py).

Tolerances are those of test_gpu_mx.py; a rounding to a 16-bit type is off by
half a step, relative to the value or, below the type's smallest normal number,
of its subnormal step.
"""
import numpy as np
import pytest
import torch

import quantized_moe_expert_top_amd as q
from oracle import mx_oracle as mx
from tests.test_gpu_mx import (DEV, DT, FMT, NORM, Product, check_product, check_route, close, decoded, dev, f64,
                               layer_reference, show)

pytestmark = pytest.mark.gpu


# --------------------------------------------------------------------- routing
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("gt", [1, 2])
@pytest.mark.parametrize("E,G,tg,k", [(16, 4, 2, 4), (16, 4, 1, 3), (16, 4, 4, 5), (60, 5, 2, 6), (256, 8, 4, 8),
                                      (512, 64, 3, 7)])
def test_route_groups_of_unbounded_bias(sigmoid, gt, E, G, tg, k):
    """A bias of +inf in every group, in two experts of every group, in some groups: ties between groups go to the
    lower one."""
    rng = np.random.default_rng(E + G + gt)
    logits = rng.standard_normal((9, E)).astype(np.float32)
    logits[3, ::2] = -np.inf
    size = E // G
    for firsts, groups in ((1, range(G)), (2, range(G)), (1, range(1, G, 2)), (2, range(G - 1, G))):
        bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
        for g in groups:
            bias[g * size: g * size + firsts] = np.inf
        check_route(logits, k, sigmoid=sigmoid, bias=bias, n_group=G, topk_group=tg, group_top=gt)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("gt", [1, 2])
@pytest.mark.parametrize("low,high", [(2.5e38, 3.4e38), (-3.4e38, -2.5e38), (-3.4e38, 3.4e38)])
@pytest.mark.parametrize("E,G,tg,k", [(16, 4, 2, 4), (96, 6, 5, 9), (256, 8, 3, 8)])
def test_route_groups_of_huge_biases(sigmoid, gt, low, high, E, G, tg, k):
    """Finite biases whose sums of two pass the largest float32: groups by their float64 sums."""
    rng = np.random.default_rng(E + G + gt)
    logits = rng.standard_normal((7, E)).astype(np.float32)
    logits[2, 1::2] = np.nan
    bias = rng.uniform(low, high, E).astype(np.float32)
    check_route(logits, k, sigmoid=sigmoid, bias=bias, n_group=G, topk_group=tg, group_top=gt)
    bias[: E // G] = 0.25  # one ordinary group
    check_route(logits, k, sigmoid=sigmoid, bias=bias, n_group=G, topk_group=tg, group_top=gt)


# -------------------------------------------------------------------- the norm
def norm_rows(rng, kind, rows, H):
    """Rows and weights whose products, or whose norm's factor, leave float32's normal range, with finite norms."""
    x, w = rng.standard_normal((rows, H)), 1 + 0.2 * rng.standard_normal(H)
    if kind == "products past the largest":   # v * w up to 2^129, norms near 2
        return np.clip(x, -3, 3) * 2.0 ** 125, w * 2
    if kind == "products below the smallest":
        return x * 1e-20, w * 1e-19
    if kind == "subnormal rows":
        return x * 2.0 ** -130, w
    if kind == "subnormal rows, large weights":
        return x * 2.0 ** -130, w * 2.0 ** 100
    if kind == "largest rows":                # a factor below the smallest normal number
        return np.where(rng.random((rows, H)) < 0.5, 1.0, -1.0) * rng.uniform(0.6, 1.0, (rows, H)) * 3.3e38, w
    if kind == "far apart in a row":          # large weights bring small values back
        e = rng.integers(-90, 91, (rows, H))
        e[:, 0] = 90
        return x * np.exp2(e.astype(float)), np.where(rng.random(H) < 0.5, w, w * 2.0 ** 120)
    if kind == "norms below the smallest":
        return x, w * np.exp2(-rng.integers(120, 150, H).astype(float))
    raise KeyError(kind)


@pytest.mark.parametrize("kind", ["products past the largest", "products below the smallest", "subnormal rows",
                                  "subnormal rows, large weights", "largest rows", "far apart in a row",
                                  "norms below the smallest"])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,H", [(3, 96), (5, 2048), (600, 4096), (2, 16384)])
def test_rmsnorm_ends_of_the_range(kind, dt, rows, H):
    rng = np.random.default_rng(H + rows)
    x, w = (dev(a.astype(np.float32), DT[dt]) for a in norm_rows(rng, kind, rows, H))
    show("norm", kind, dt, rows, H)
    n = mx.rmsnorm(f64(x), f64(w), 0.0)
    assert np.isfinite(n).all() and np.abs(n).max() < 2.0 ** 127.9
    info = torch.finfo(DT[dt])
    for fmt in ("e4m3", "e2m1"):
        o = q.moe_rmsnorm_mx(x, w, 0.0, fmt=FMT[fmt], want_y=True)
        step = info.tiny * info.eps  # of subnormal numbers
        close(f64(o.y), n, (info.eps / 2 + NORM) * np.abs(n) + step / 2 * (1 + NORM), "y")
        assert np.array_equal(decoded(o.rows), mx.values(*mx.quantize(n, FMT[fmt]), FMT[fmt]))


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_rmsnorm_past_the_largest(dt):
    """Norms past the largest float32 are infinite: y has that infinity, the block is not a number; others stay."""
    x = torch.ones(2, 128, device=DEV, dtype=DT[dt])
    x[1, 5] = -1
    w = torch.ones(128, device=DEV, dtype=DT[dt])
    w[5] = 3.3e38
    x[:, 5] *= 4  # mean square 1.12: the norm there 4 / 1.06 * 3.3e38
    o = q.moe_rmsnorm_mx(x, w, 0.0, want_y=True)
    y = f64(o.y)
    assert y[0, 5] == np.inf and y[1, 5] == -np.inf and np.isfinite(np.delete(y, 5, 1)).all()
    assert (o.rows.scales[:, 0] == 255).all() and (o.rows.scales[:, 1:] != 255).all()


# ----------------------------------------------------------------- the product
def sparse_counts(E, rng):
    """Rows of E experts: mostly none, one or several row tiles next to the multiples of 64 and at the ends."""
    c = np.zeros(E, int)
    for e in (0, 3, 62, 63, 64, 65, 126, 127, 128, 129, 191, 192, 511, 640, 959, 960, E - 2, E - 1):
        if 0 <= e < E:
            c[e] = rng.choice([0, 1, 31, 64, 65, 129, 200])
    c[min(E - 1, 64)] = 130
    return [int(v) for v in c]


MANY = [("e4m3", q.MOE_KERNEL_SMALL), ("e4m3", q.MOE_KERNEL_TILE64), ("e4m3", q.MOE_KERNEL_TILE128),
        ("e2m1", q.MOE_KERNEL_TILE64), ("e2m1", q.MOE_KERNEL_TILE128), ("e2m1", q.MOE_KERNEL_TILE64_SPLIT_K)]


@pytest.mark.parametrize("act,kernel", MANY)
@pytest.mark.parametrize("E,N,K", [(64, 320, 384), (65, 320, 384), (128, 64, 384), (130, 320, 512), (1000, 64, 384),
                                   (1024, 64, 384)])
def test_product_many_experts(act, kernel, E, N, K):
    """Tiles found over several groups of 64 segments, against float64."""
    p = Product(E + N, E, N, K, act, sparse_counts(E, np.random.default_rng(E)), k=2)
    check_product(p, q.MOE_EPI_NONE_F32, kernel, f"{act} {E} experts {N}x{K}")
    check_product(p, q.MOE_EPI_SWIGLU_E4M3, kernel, f"{act} {E} experts {N}x{K}")


@pytest.mark.parametrize("act,kernel", MANY)
def test_product_of_blocks_that_are_not_numbers(act, kernel):
    """Blocks as the quantisation leaves them for an infinity or NaN (scale byte 255, codes 0), in rows and in weights:
    the whole row, the expert's channel."""
    E, N, K = 2, 64, 512
    g = torch.Generator(device=DEV).manual_seed(4)
    wv, xv = torch.randn(E, N, K, device=DEV, generator=g), torch.randn(150, K, device=DEV, generator=g)
    wv[1, 33, 200], xv[7, 450], xv[100, 3] = float("inf"), float("nan"), float("-inf")
    w = q.moe_mx_repack(q.mx_experts(q.moe_quantize_mx(wv, q.MOE_MX_E2M1)))
    a = q.moe_quantize_mx(xv, FMT[act])
    show("not numbers", act, kernel)
    y = q.moe_grouped_mxgemm(w, a, dev(np.array([0, 90, 150], np.int32)), 150, q.MOE_EPI_NONE_F32, kernel=kernel)
    want = torch.zeros(150, N, dtype=torch.bool, device=DEV)
    want[7], want[100] = True, True
    want[90:, 33] = True
    assert torch.equal(torch.isnan(y), want)
    h = q.moe_grouped_mxgemm(w, a, dev(np.array([0, 90, 150], np.int32)), 150, q.MOE_EPI_SWIGLU_E4M3, kernel=kernel)
    bad = torch.zeros(150, 1, dtype=torch.bool, device=DEV)
    bad[7], bad[100], bad[90:] = True, True, True
    assert torch.equal(h.scales == 255, bad)


# ------------------------------------------------------------------- the layer
def test_layer_outputs_past_float16():
    """Expert outputs past 65504: finite where they travel to the combine as float32 or bfloat16, infinite as float16
    (the default), as the documentation says."""
    T, E, H, I, k = 20, 4, 128, 256, 2
    rng = np.random.default_rng(2)
    g = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
    gu = q.moe_quantize_mx(dev(2 * g(E, 2 * I, H)), q.MOE_MX_E2M1)
    dn = q.moe_quantize_mx(dev(64 * g(E, H, I)), q.MOE_MX_E2M1)
    x, logits = q.moe_quantize_mx(dev(g(T, H))), g(T, E)
    _, _, ref, _ = layer_reference(decoded(x), logits, k, decoded(gu), decoded(dn), mx.E4M3, {})
    assert np.abs(ref).max() > 2 * 65504
    t13, t2 = (q.moe_mx_repack(q.mx_experts(v)) for v in (gu, dn))
    for y_dtype in (torch.float32, torch.bfloat16, torch.float16):
        show("past float16", y_dtype)
        buf = q.alloc_mx_layer(T, E, k, H, I, DEV, y_dtype=y_dtype)
        out = f64(q.moe_mx_layer_forward(x, dev(logits), k, t13, t2, buf=buf).out)
        if y_dtype == torch.float16:
            assert np.isinf(f64(buf.y_perm)).any()
        else:
            assert np.isfinite(out).all()
            assert np.linalg.norm(out - ref) <= 5e-3 * np.linalg.norm(ref)


# ------------------------------------------------------- the calls of README.md
README_CALLS = """\
w13 = q.moe_mx_repack(q.mx_experts(q.moe_quantize_mx(gate_up, q.MOE_MX_E2M1)))   # [E][2I][H]: gate rows, then up rows
w2 = q.moe_mx_repack(q.mx_experts(q.moe_quantize_mx(down, q.MOE_MX_E2M1)))       # [E][H][I]
n = q.moe_rmsnorm_mx(x, norm_weight, 1e-5, residual=residual, fmt=q.MOE_MX_E4M3) # n.rows feeds the experts
routing = q.ScoredRouting(score=q.MOE_SCORE_SIGMOID, bias=bias)
out = q.moe_mx_layer_forward(n.rows, logits, k, w13, w2, routing).out            # bf16 [T][H]
"""


def test_calls_that_the_readme_shows():
    T, E, H, I, k = 12, 4, 256, 128, 2
    r = lambda *s: torch.randn(*s, device=DEV)  # noqa: E731
    names = dict(q=q, x=r(T, H).bfloat16(), residual=r(T, H).bfloat16(), norm_weight=r(H).bfloat16(), logits=r(T, E),
                 bias=r(E), k=k, gate_up=r(E, 2 * I, H).bfloat16(), down=r(E, H, I).bfloat16())
    exec(README_CALLS, names)  # noqa: S102
    out = names["out"]
    assert isinstance(out, torch.Tensor) and out.shape == (T, H) and out.dtype == torch.bfloat16
    assert torch.isfinite(out).all() and out.abs().sum() > 0
