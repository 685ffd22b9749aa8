"""GPU checks of the experts in 16 bits, their gradients and the low-rank
adapters against float64 references (oracle/dense_oracle.py).

Tolerances.  A sum of n products of 16-bit numbers (exact in fp32) accumulated
in fp32 is off by at most n * 2^-23 times the sum of their magnitudes m,
whatever the order and also if an addition inside a matrix instruction is cut
and not rounded (2^-23 of each partial sum, none of which exceeds m).  An
output's rounding adds half a step: 2^-8 (bf16), 2^-11 (fp16), 2^-24 (fp32)
relative, and half the smallest subnormal (2^-25 in fp16).  `bound` is that;
the SwiGLU's derivatives carry the sums' errors on, and its exponential,
reciprocal and products add 2^-19 (gates down to -16; the gates here stay above
-12).
"""
import itertools

import numpy as np
import pytest
import torch

import quantized_moe_expert_top_amd as q
from oracle import dense_oracle as do

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
TINY = {"bf16": 0.0, "fp16": 2.0 ** -25, "fp32": 0.0}
EPI = {"bf16": q.MOE_EPI_NONE, "fp16": q.MOE_EPI_NONE_F16, "fp32": q.MOE_EPI_NONE_F32}
KERNELS = {"auto": q.MOE_KERNEL_AUTO, "small": q.MOE_KERNEL_SMALL, "128": q.MOE_KERNEL_TILE128,
           "256": q.MOE_KERNEL_TILE256}
TILES = {name: kr for name, kr in KERNELS.items() if name != "small"}  # what runs the weights' gradient
SWIGLU = 2.0 ** -19


def f64(t):
    return t.double().cpu().numpy()


def dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV).to(dtype)


def i32(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def close(got, ref, tol, what=""):
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off, first at {np.argwhere(bad)[0]}: " \
        f"{got[bad][0]} for {ref[bad][0]} (tolerance {np.broadcast_to(tol, ref.shape)[bad][0]})"


def bound(ref, mag, n, dt):
    return HALF[dt] * np.abs(ref) * (1 + 2.0 ** -20) + TINY[dt] + (n + 2) * 2.0 ** -23 * mag


def swiglu_bound(y, mag, n, dt):
    """silu(g) u with both sums off: |silu'| <= 1.1."""
    g, u = np.split(y, 2, axis=1)
    eg, eu = np.split((n + 2) * 2.0 ** -23 * mag, 2, axis=1)
    h = do.swiglu(y)
    return (HALF[dt] + SWIGLU) * np.abs(h) + TINY[dt] + 1.1 * eg * (np.abs(u) + eu) + np.abs(g * do.sigmoid(g)) * eu


def swiglu_grad_bound(dh, err, pre, dt):
    out = do.swiglu_grad(np.abs(dh), pre)
    e = do.swiglu_grad(err, pre)
    # each of the factors s, 1 - s, g s (1 - s) and 1 is at most 1.1 and computed to 2^-19 of its terms
    g, u = np.split(np.abs(pre), 2, axis=1)
    own = np.concatenate([np.abs(dh) * u * (1 + g), np.abs(dh) * g], axis=1) * 2.0 ** -21
    return HALF[dt] * (np.abs(out) + np.abs(e)) * 1.01 + TINY[dt] + np.abs(e) + own


def tile(kr):
    """The kernel choice of a weights' gradient beside products by `kr`."""
    return q.MOE_KERNEL_AUTO if kr == q.MOE_KERNEL_SMALL else kr


class Batch:
    """Rows of uneven segments: `counts` rows per expert; with k > 1 they are gathered from tokens."""

    def __init__(self, seed, counts, N, K, dt, k=1, gather=False, before=0, after=0):
        r = np.random.default_rng(seed)
        self.E, self.N, self.K, self.k = len(counts), N, K, k
        self.offsets = before + np.concatenate([[0], np.cumsum(counts)])
        self.M = int(self.offsets[-1]) + after
        self.seg = i32(self.offsets)
        self.w = dev(r.standard_normal((self.E, N, K)) / np.sqrt(K), DT[dt])
        rows = self.M
        if gather:
            rows = -(-self.M // k) + 3
            self.pairs_np = r.permutation(rows * k)[: self.M]
            self.pairs = i32(self.pairs_np)
            self.src = self.pairs_np // k
        else:
            self.pairs, self.src = None, np.arange(self.M)
        self.a = dev(r.standard_normal((max(rows, 1), K)), DT[dt])
        self.dy = dev(r.standard_normal((max(self.M, 1), N)), DT[dt])[: self.M]
        self.rows = f64(self.a)[self.src]  # grouped
        self.live = np.zeros(self.M, bool)
        self.live[before : int(self.offsets[-1])] = True


UNEVEN = [0, 1, 33, 0, 129, 15, 300, 64]
SIZES = [  # counts, N, K
    ([1], 16, 8), ([3, 0, 2], 48, 72), (UNEVEN, 272, 200), ([257, 16, 17, 1], 528, 1032), ([70, 31, 256], 640, 320)]


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("size", range(len(SIZES)))
def test_product(lib, size, dt, kernel):
    counts, N, K = SIZES[size]
    for gather, epi in itertools.product((False, True), ("bf16", "fp16", "fp32", "swiglu", "swiglu_pre")):
        b = Batch(size, counts, N, K, dt, k=3 if gather else 1, gather=gather)
        y, mag = do.product(f64(b.w), b.rows, b.offsets)
        args = dict(gather_pair=b.pairs, k=b.k, kernel=KERNELS[kernel])
        if epi in EPI:
            got = q.moe_grouped_gemm(b.w, b.a, b.seg, b.M, EPI[epi], **args)
            assert got.dtype == DT[epi] and got.shape == (b.M, N)
            close(f64(got), y, bound(y, mag, K, epi), f"{epi} gather {gather}")
            continue
        pre = torch.empty(b.M, N, dtype=DT[dt], device=DEV) if epi == "swiglu_pre" else None
        got = q.moe_grouped_gemm(b.w, b.a, b.seg, b.M, q.MOE_EPI_SWIGLU, pre=pre, **args)
        assert got.dtype == DT[dt] and got.shape == (b.M, N // 2)
        close(f64(got), do.swiglu(y), swiglu_bound(y, mag, K, dt), f"{epi} gather {gather}")
        if pre is not None:
            close(f64(pre), y, bound(y, mag, K, dt), f"pre gather {gather}")


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("size", range(len(SIZES)))
def test_grad_rows(lib, size, dt, kernel):
    counts, N, K = SIZES[size]
    b = Batch(size, counts, N, K, dt)
    ref, mag = do.grad_rows(f64(b.w), f64(b.dy), b.offsets)
    for epi in EPI:
        got = q.moe_grouped_gemm_grad_rows(b.w, b.dy, b.seg, b.M, EPI[epi], kernel=KERNELS[kernel])
        assert got.dtype == DT[epi] and got.shape == (b.M, K)
        close(f64(got), ref, bound(ref, mag, N, epi), epi)
    pre = dev(np.random.default_rng(9).standard_normal((b.M, 2 * K)) * 2, DT[dt])
    got = q.moe_grouped_gemm_grad_rows(b.w, b.dy, b.seg, b.M, q.MOE_EPI_SWIGLU_GRAD, pre=pre, kernel=KERNELS[kernel])
    assert got.dtype == DT[dt] and got.shape == (b.M, 2 * K)
    close(f64(got), do.swiglu_grad(ref, f64(pre)),
          swiglu_grad_bound(ref, (N + 2) * 2.0 ** -23 * mag, f64(pre), dt), "swiglu_grad")


@pytest.mark.parametrize("kernel", TILES)
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("size", range(len(SIZES)))
def test_grad_weights(lib, size, dt, kernel):
    counts, N, K = SIZES[size]
    for gather, epi in itertools.product((False, True), EPI):
        b = Batch(size, counts, N, K, dt, k=3 if gather else 1, gather=gather)
        ref, mag = do.grad_weights(f64(b.dy), b.rows, b.offsets)
        got = q.moe_grouped_gemm_grad_weights(b.dy, b.a, b.seg, b.E, b.M, EPI[epi], gather_pair=b.pairs, k=b.k,
                                              kernel=KERNELS[kernel])
        assert got.dtype == DT[epi] and got.shape == (b.E, N, K)
        n = np.array(counts).reshape(-1, 1, 1)
        close(f64(got), ref, bound(ref, mag, n, epi), f"{epi} gather {gather}")


@pytest.mark.parametrize("counts,N,K", [([5000], 64, 40), ([0, 2100, 3], 72, 136), ([9000, 1], 16, 16)])
def test_grad_weights_long_segments(lib, counts, N, K):
    """Few weights, many rows: the rows are split over workgroups (with a workspace)."""
    for gather in (False, True):
        b = Batch(3, counts, N, K, "bf16", k=2 if gather else 1, gather=gather)
        ref, mag = do.grad_weights(f64(b.dy), b.rows, b.offsets)
        n = np.array(counts).reshape(-1, 1, 1)
        for kernel in TILES.values():
            ws = torch.full((q.moe_grouped_gemm_grad_weights_workspace_size(b.E, N, K, b.M, kernel),), 255,
                            dtype=torch.uint8, device=DEV)  # NaNs
            got = q.moe_grouped_gemm_grad_weights(b.dy, b.a, b.seg, b.E, b.M, gather_pair=b.pairs, k=b.k, kernel=kernel,
                                                  workspace=ws if ws.numel() else None)
            close(f64(got), ref, bound(ref, mag, n, "fp32"))


@pytest.mark.parametrize("kernel", KERNELS)
def test_rows_of_no_segment_are_left(lib, kernel):
    """A slice of a longer offset table: rows before and behind it are neither written nor read."""
    kr = KERNELS[kernel]
    b = Batch(5, [0, 40, 3, 0, 130], 80, 104, "bf16", before=37, after=19)
    dead = torch.from_numpy(~b.live).to(DEV)
    b.dy[dead] = float("nan")
    a = b.a.clone()
    a[dead] = float("nan")
    for shape, call in (
            ((b.M, 80), lambda o: q.moe_grouped_gemm(b.w, a, b.seg, b.M, out=o, kernel=kr)),
            ((b.M, 40), lambda o: q.moe_grouped_gemm(b.w, a, b.seg, b.M, q.MOE_EPI_SWIGLU, out=o, kernel=kr)),
            ((b.M, 104), lambda o: q.moe_grouped_gemm_grad_rows(b.w, b.dy, b.seg, b.M, out=o, kernel=kr))):
        out = torch.full(shape, 7.0, dtype=torch.bfloat16, device=DEV)
        call(out)
        assert (out[dead] == 7).all() and not (out[~dead] == 7).all()
        assert torch.isfinite(out).all()
    dw = q.moe_grouped_gemm_grad_weights(b.dy, a, b.seg, b.E, b.M, kernel=tile(kr))
    live = np.where(b.live[:, None], 1, 0)
    ref, mag = do.grad_weights(np.where(live, f64(b.dy), 0), np.where(live, b.rows, 0), b.offsets)
    close(f64(dw), ref, bound(ref, mag, 130, "fp32"))
    assert (dw[0] == 0).all() and (dw[3] == 0).all()


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_not_finite_values_stay_in_their_rows(lib, kernel, bad):
    """A row that is not a number reaches its own outputs only, and an expert's its own rows (K = 72 and N = 80: the
    last step of each sum ends inside a tile)."""
    kr = KERNELS[kernel]
    b = Batch(6, [20, 1, 70], 80, 72, "bf16")
    y, mag = do.product(f64(b.w), b.rows, b.offsets)
    b.a[20] = bad
    got = f64(q.moe_grouped_gemm(b.w, b.a, b.seg, b.M, kernel=kr))
    ok = np.arange(b.M) != 20
    close(got[ok], y[ok], bound(y, mag, 72, "bf16")[ok])
    assert not np.isfinite(got[20]).any()
    da, dmag = do.grad_rows(f64(b.w), f64(b.dy), b.offsets)
    dy = b.dy.clone()
    dy[20] = bad
    got = f64(q.moe_grouped_gemm_grad_rows(b.w, dy, b.seg, b.M, kernel=kr))
    close(got[ok], da[ok], bound(da, dmag, 80, "bf16")[ok])
    assert not np.isfinite(got[20]).any()
    # its weights' gradient alone is lost; the experts beside it keep theirs
    got = f64(q.moe_grouped_gemm_grad_weights(dy, b.a, b.seg, b.E, b.M, kernel=tile(kr)))
    ref, wmag = do.grad_weights(f64(b.dy), b.rows, b.offsets)
    for e in (0, 2):
        close(got[e], ref[e], bound(ref, wmag, 70, "fp32")[e])
    assert not np.isfinite(got[1]).any()
    # an expert whose weights are not numbers: its rows only
    w = b.w.clone()
    w[0] = bad
    a = Batch(6, [20, 1, 70], 80, 72, "bf16").a
    got = f64(q.moe_grouped_gemm(w, a, b.seg, b.M, kernel=kr))
    close(got[20:], y[20:], bound(y, mag, 72, "bf16")[20:])
    assert not np.isfinite(got[:20]).any()


def test_swiglu_ends_of_the_range(lib):
    """Gates far out: silu is 0 below and the gate itself above, its derivative 0 and 1; no NaN from exp's overflow."""
    K = 8
    g = np.array([-1000, -200, -90, -30, 0, 30, 90, 1000.0])
    w = np.zeros((1, 16, K))
    w[0, :8] = np.diag(g)
    w[0, 8:] = np.eye(K) * 2
    a = torch.ones(1, K, dtype=torch.bfloat16, device=DEV)
    out = f64(q.moe_grouped_gemm(dev(w, torch.bfloat16), a, i32([0, 1]), 1, q.MOE_EPI_SWIGLU))[0]
    np.testing.assert_allclose(out, np.where(g > 0, 2 * f64(dev(g, torch.bfloat16)), 0), atol=1e-10, rtol=2.0 ** -8)
    pre = dev(np.concatenate([g, np.full(8, 2.0)])[None], torch.bfloat16)
    eye = torch.eye(8, dtype=torch.bfloat16, device=DEV)[None]
    d = f64(q.moe_grouped_gemm_grad_rows(eye, a, i32([0, 1]), 1, q.MOE_EPI_SWIGLU_GRAD, pre=pre))[0]
    np.testing.assert_allclose(d[:8], np.where(g > 0, 2.0, np.where(g == 0, 1.0, 0.0)), atol=1e-10, rtol=2.0 ** -8)
    np.testing.assert_allclose(d[8:], np.where(g > 0, f64(dev(g, torch.bfloat16)), 0), atol=1e-10, rtol=2.0 ** -8)


def test_results_repeat_bit_for_bit(lib):
    b = Batch(7, [300, 0, 45, 2000], 136, 264, "bf16", k=4, gather=True)
    for kr in KERNELS.values():
        calls = (lambda: q.moe_grouped_gemm(b.w, b.a, b.seg, b.M, gather_pair=b.pairs, k=4, kernel=kr),
                 lambda: q.moe_grouped_gemm_grad_rows(b.w, b.dy, b.seg, b.M, kernel=kr),
                 lambda: q.moe_grouped_gemm_grad_weights(b.dy, b.a, b.seg, b.E, b.M, gather_pair=b.pairs, k=4, kernel=tile(kr)))
        for f in calls:
            first = f()
            for _ in range(4):
                assert torch.equal(first, f())


def test_more_experts_than_lanes(lib):
    """200 experts, most without rows, tiles found over several groups of 64 segments."""
    counts = np.zeros(200, int)
    counts[[0, 63, 64, 127, 130, 199]] = [5, 40, 1, 300, 0, 17]
    b = Batch(8, counts, 48, 40, "fp16", k=2, gather=True)
    y, mag = do.product(f64(b.w), b.rows, b.offsets)
    da, dmag = do.grad_rows(f64(b.w), f64(b.dy), b.offsets)
    dw, wmag = do.grad_weights(f64(b.dy), b.rows, b.offsets)
    for kr in KERNELS.values():
        close(f64(q.moe_grouped_gemm(b.w, b.a, b.seg, b.M, q.MOE_EPI_NONE_F32, gather_pair=b.pairs, k=2, kernel=kr)), y,
              bound(y, mag, 40, "fp32"))
        close(f64(q.moe_grouped_gemm_grad_rows(b.w, b.dy, b.seg, b.M, q.MOE_EPI_NONE_F32, kernel=kr)), da,
              bound(da, dmag, 48, "fp32"))
        close(f64(q.moe_grouped_gemm_grad_weights(b.dy, b.a, b.seg, 200, b.M, gather_pair=b.pairs, k=2, kernel=tile(kr))), dw,
              bound(dw, wmag, 300, "fp32"))


@pytest.mark.parametrize("kernel", KERNELS)
def test_offsets_past_32_bits(lib, kernel):
    """More than 2^32 bytes of rows, outputs, gradients and pre-activations: the last rows are right."""
    kr = KERNELS[kernel]
    M, N, K = 300_001, 8192, 8
    g = torch.Generator(device=DEV).manual_seed(3)
    w = torch.randn(2, N, K, generator=g, device=DEV).bfloat16()
    a = torch.randn(M, K, generator=g, device=DEV).bfloat16()
    seg = i32([0, 7, M])
    out = q.moe_grouped_gemm(w, a, seg, M, kernel=kr)
    at = slice(M - 70, M)
    ref = f64(a[at]) @ f64(w[1]).T
    mag = np.abs(f64(a[at])) @ np.abs(f64(w[1])).T
    close(f64(out[at]), ref, bound(ref, mag, K, "bf16"))
    # the same rows back: dy is past 4 GiB now
    da = q.moe_grouped_gemm_grad_rows(w, out, seg, M, q.MOE_EPI_NONE_F32, kernel=kr)
    ref = f64(out[at]) @ f64(w[1])
    mag = np.abs(f64(out[at])) @ np.abs(f64(w[1]))
    close(f64(da[at]), ref, bound(ref, mag, N, "fp32"))
    out[:-33] = 0
    dw = q.moe_grouped_gemm_grad_weights(out, a, seg, 2, M, kernel=tile(kr))
    ref = f64(out[-33:]).T @ f64(a[-33:])
    mag = np.abs(f64(out[-33:])).T @ np.abs(f64(a[-33:]))
    close(f64(dw[1]), ref, bound(ref, mag, M, "fp32"))
    assert (dw[0] == 0).all()


def test_product_for_an_empty_batch(lib):
    w = torch.zeros(2, 16, 8, dtype=torch.bfloat16, device=DEV)
    none, seg = torch.empty(0, 8, dtype=torch.bfloat16, device=DEV), i32([0, 0, 0])
    assert q.moe_grouped_gemm(w, none, seg, 0).shape == (0, 16)
    dy = torch.empty(0, 16, dtype=torch.bfloat16, device=DEV)
    assert q.moe_grouped_gemm_grad_rows(w, dy, seg, 0).shape == (0, 8)
    dw = q.moe_grouped_gemm_grad_weights(dy, none, seg, 2, 0, out=torch.ones(2, 16, 8, device=DEV))
    assert (dw == 0).all()


# ------------------------------------------------------ the combine's gradient
@pytest.mark.parametrize("T,k,E,H", [(1, 1, 1, 8), (5, 3, 7, 264), (33, 8, 64, 2048), (3, 20, 40, 4104)])
@pytest.mark.parametrize("y_dt", ["bf16", "fp16", "fp32"])
def test_combine_grad(lib, T, k, E, H, y_dt):
    r = np.random.default_rng(T)
    ids = np.stack([r.permutation(E)[:k] for _ in range(T)])
    ids[r.random(ids.shape) < 0.2] = -1
    ids[0, 0] = E + 5
    p = q.moe_permute(i32(ids), E)
    nv = int(p.seg_offsets[-1])
    pos = p.pair_pos.cpu().numpy().reshape(T, k)
    y = dev(r.standard_normal((T * k, H)), DT[y_dt])
    dout = dev(r.standard_normal((T, H)), torch.bfloat16)
    w = torch.softmax(dev(r.standard_normal((T, k)), torch.float32), -1)
    y[p.pair_pos[p.pair_pos >= nv].long()] = float("nan")  # rows that nothing wrote
    yz = np.nan_to_num(f64(y))
    dy, dw, mag, dl = do.combine_grad(f64(dout), yz, pos, f64(w), nv, ids, E)
    for dt in ("bf16", "fp16"):
        buf = torch.full((T * k, H), 7.0, dtype=DT[dt], device=DEV)
        g = q.moe_unpermute_combine_grad(dout, y, p.pair_pos, w, T, k, dtype=DT[dt], dy=buf, ids=i32(ids), E=E,
                                         n_valid=p.seg_offsets[-1:])
        # w * dout: the product's rounding in fp32, then the output's
        close(f64(g.dy[:nv]), dy[:nv], (HALF[dt] + 2.0 ** -23) * np.abs(dy[:nv]) + TINY[dt])
        assert (g.dy[nv:] == 7).all()
        e_dw = (H + 2) * 2.0 ** -23 * mag
        close(f64(g.dw), dw, e_dw)
        # every term of a logit's gradient carries its dw's error and some roundings of what it multiplies
        amp = np.abs(f64(w)) * (np.abs(dw) + (np.abs(f64(w)) * np.abs(dw)).sum(1, keepdims=True))
        err = np.abs(f64(w)) * (e_dw + (np.abs(f64(w)) * e_dw).sum(1, keepdims=True)) + (k + 4) * 2.0 ** -23 * amp
        tol = np.zeros((T, E))
        for t in range(T):
            for j in range(k):
                if 0 <= ids[t, j] < E:
                    tol[t, ids[t, j]] += err[t, j]
        close(f64(g.dlogits), dl, tol)
    one = q.moe_unpermute_combine_grad(dout, y, p.pair_pos, None, T, k, n_valid=p.seg_offsets[-1:])
    assert one.dlogits is None
    assert torch.equal(one.dy[:nv], dout[torch.div(p.sorted_pair[:nv], k, rounding_mode="floor").long()])


def test_combine_grad_of_weights_without_rows(lib):
    """The weight of a pair without an expert may be anything: it reaches no gradient."""
    ids = i32([[1, -1, 2], [0, 2, 7]])
    p = q.moe_permute(ids, 3)
    r = np.random.default_rng(8)
    y, dout = dev(r.standard_normal((6, 24)), torch.float32), dev(r.standard_normal((2, 24)), torch.bfloat16)
    grads = []
    for v in (0.0, float("nan"), float("inf")):
        w = dev([[0.5, v, 0.5], [0.25, 0.75, v]], torch.float32)
        g = q.moe_unpermute_combine_grad(dout, y, p.pair_pos, w, 2, 3, ids=ids, E=3, n_valid=p.seg_offsets[-1:])
        grads.append((g.dy[:4], g.dw, g.dlogits))
    for g in grads:
        assert all(torch.isfinite(t).all() and torch.equal(t, u) for t, u in zip(g, grads[0]))


def test_combine_grad_by_differences(lib):
    """The logits' and outputs' gradients against central differences of <dout, combine(softmax gates)> in float64."""
    T, k, E, H = 4, 3, 6, 64
    r = np.random.default_rng(1)
    logits = r.standard_normal((T, E)).astype(np.float32)
    ids, w, p = q.moe_route_permute(dev(logits, torch.float32), k)
    y, dout = dev(r.standard_normal((T * k, H)), torch.float32), dev(r.standard_normal((T, H)), torch.bfloat16)
    g = q.moe_unpermute_combine_grad(dout, y, p.pair_pos, w, T, k, ids=ids, E=E)
    idn, pos = ids.cpu().numpy(), p.pair_pos.cpu().numpy().reshape(T, k)

    def loss(lg, yv):
        s = 0.0
        for t in range(T):
            e = np.exp(lg[t, idn[t]] - lg[t, idn[t]].max())
            s += f64(dout)[t] @ ((e / e.sum())[:, None] * yv[pos[t]]).sum(0)
        return s

    y64, l64, h = f64(y), logits.astype(np.float64), 1e-5
    for t in range(T):
        for e in range(E):
            d = np.zeros_like(l64)
            d[t, e] = h
            want = (loss(l64 + d, y64) - loss(l64 - d, y64)) / (2 * h)
            assert abs(float(g.dlogits[t, e]) - want) <= 1e-5 * (1 + abs(want))
    for i in range(0, T * k, 5):
        d = np.zeros_like(y64)
        d[i, 3] = h
        want = (loss(l64, y64 + d) - loss(l64, y64 - d)) / (2 * h)
        assert abs(float(g.dy[i, 3]) - want) <= (2.0 ** -8 + 1e-5) * abs(want) + 1e-6


# --------------------------------------------------------------------- adapters
def adapter_batch(seed, ids, n, r, K, N, dt, y_dt):
    g = np.random.default_rng(seed)
    T = len(ids)
    mk = lambda *s: g.standard_normal(s)  # noqa: E731
    x, y = dev(mk(T, K), DT[dt]), dev(mk(T, N), DT[y_dt])
    A, B = dev(mk(n, r, K) / np.sqrt(K), DT[dt]), dev(mk(n, N, r), DT[dt])
    scale = dev(0.5 + g.random(n), torch.float32)
    return x, y, A, B, scale, q.moe_permute(i32(ids).view(T, 1), n)


def adapter_bound(ref, y, mag, K, r, dt, y_dt):
    """Both sums' errors, v as two 16-bit numbers (2^-16 in bf16, 2^-22 in fp16, of its magnitude), out's rounding."""
    split = 2.0 ** -16 if dt == "bf16" else 2.0 ** -21
    return HALF[y_dt] * np.abs(ref) * (1 + 2.0 ** -20) + TINY[y_dt] + mag * ((K + 2 * r + 8) * 2.0 ** -23 + split)


ADAPTER_IDS = {
    "one": [2], "none": [-1, -1, 7], "each": list(range(7)), "mixed": [3] * 40 + [-1] * 3 + [0] + [3] * 30 + [5] * 33 + [9],
    "alternating": [i % 3 - 1 for i in range(150)]}


@pytest.mark.parametrize("r,K,N", [(8, 16, 8), (16, 1032, 264), (24, 512, 1000), (64, 264, 520), (128, 136, 72)])
@pytest.mark.parametrize("which", ADAPTER_IDS)
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_adapters(lib, which, r, K, N, dt):
    ids, n = ADAPTER_IDS[which], 7
    for y_dt in ("bf16", "fp16", "fp32"):
        x, y, A, B, scale, p = adapter_batch(r, ids, n, r, K, N, dt, y_dt)
        ref, mag = do.adapters(f64(y), f64(x), f64(A), f64(B), ids, f64(scale))
        got = q.moe_adapter_add(y, x, A, B, p.seg_offsets, p.sorted_pair, scale=scale)
        close(f64(got), ref, adapter_bound(ref, f64(y), mag, K, r, dt, y_dt), y_dt)
        bare = [t for t, a in enumerate(ids) if not 0 <= a < n]
        assert torch.equal(got[bare], y[bare])
        into = y.clone()
        assert q.moe_adapter_add(into, x, A, B, p.seg_offsets, p.sorted_pair, scale=scale, out=into) is into
        assert torch.equal(into, got)
        ref, mag = do.adapters(f64(y), f64(x), f64(A), f64(B), ids, np.ones(n))
        close(f64(q.moe_adapter_add(y, x, A, B, p.seg_offsets, p.sorted_pair)), ref,
              adapter_bound(ref, f64(y), mag, K, r, dt, y_dt), "scale 1")


def test_adapters_keep_to_their_tokens(lib):
    """Adapters and rows that are not numbers reach their own tokens only; tokens without an adapter are copied as they are."""
    ids = [0] * 5 + [1] * 3 + [-1] * 2 + [2] * 40
    x, y, A, B, scale, p = adapter_batch(4, ids, 3, 16, 136, 200, "bf16", "bf16")
    clean = q.moe_adapter_add(y, x, A, B, p.seg_offsets, p.sorted_pair, scale=scale)
    A[1], B[1], x[9], y[8, 0] = float("nan"), float("inf"), float("nan"), float("nan")
    got = q.moe_adapter_add(y, x, A, B, p.seg_offsets, p.sorted_pair, scale=scale)
    keep = [t for t in range(50) if t not in (5, 6, 7, 8)]
    assert torch.equal(got[keep], clean[keep])
    assert torch.isnan(got[5:8]).all() and torch.isnan(got[8, 0]) and torch.equal(got[8, 1:], y[8, 1:])


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_adapters_past_the_range(lib, dt):
    """A row or a first product that is infinite stays so (one sign), and no rank beside the given ones makes a NaN of it."""
    for r in (8, 24):
        x, A, B = dev(np.ones((2, 16)), DT[dt]), dev(np.ones((1, r, 16)), DT[dt]), dev(np.ones((1, 40, r)), DT[dt])
        y, p = dev(np.ones((2, 40)), torch.float32), q.moe_permute(i32([[0], [0]]), 1)
        x[0, 3] = -float("inf")
        got = q.moe_adapter_add(y, x, A, B, p.seg_offsets, p.sorted_pair)
        assert (got[0] == -float("inf")).all() and (got[1] == 1 + 16 * r).all()
        x[0] = 60000.0  # 16 of them: past fp16's range
        got = q.moe_adapter_add(y, x, A, B, p.seg_offsets, p.sorted_pair)
        assert (got[0] == (float("inf") if dt == "fp16" else 1 + r * 16 * float(x[0, 0]))).all() and (got[1] == 1 + 16 * r).all()


def test_adapters_beside_a_shared_projection(lib):
    """The projection by the library's product (one expert), then the adapters in place."""
    T, K, N, n, r = 45, 256, 320, 4, 16
    ids = [t % 5 - 1 for t in range(T)]
    x, _, A, B, scale, p = adapter_batch(2, ids, n, r, K, N, "bf16", "fp32")
    w = dev(np.random.default_rng(1).standard_normal((1, N, K)) / 16, torch.bfloat16)
    y = q.moe_grouped_gemm(w, x, i32([0, T]), T, q.MOE_EPI_NONE_F32)
    q.moe_adapter_add(y, x, A, B, p.seg_offsets, p.sorted_pair, scale=scale, out=y)
    base, bmag = do.product(f64(w), f64(x), [0, T])
    ref, mag = do.adapters(base, f64(x), f64(A), f64(B), ids, f64(scale))
    close(f64(y), ref, adapter_bound(ref, base, mag, K, r, "bf16", "fp32") + bound(base, bmag, K, "fp32"))


# ------------------------------------------------------------------- the layer
def layer_case(seed, T, E, k, H, I, dt):
    r = np.random.default_rng(seed)
    x = dev(r.standard_normal((T, H)), DT[dt])
    logits = dev(r.standard_normal((T, E)), torch.float32)
    gu = dev(r.standard_normal((E, 2 * I, H)) / np.sqrt(H), DT[dt])
    dn = dev(r.standard_normal((E, H, I)) / np.sqrt(I), DT[dt])
    dout = dev(r.standard_normal((T, H)), torch.bfloat16)
    return x, logits, gu, dn, dout


def layer_reference(x, logits, gu, dn, k, dout):
    """Output and gradients by float64 automatic differentiation, experts chosen on the logits (CPU)."""
    v = [t.double().cpu().requires_grad_() for t in (x, logits, gu, dn)]
    xx, lg, wg, wd = v
    top = lg.topk(k, -1)
    gate = torch.softmax(top.values, -1)
    out = torch.zeros(x.shape[0], dn.shape[1], dtype=torch.float64)
    I = dn.shape[2]
    for j in range(k):
        rows = []
        for t in range(x.shape[0]):
            e = int(top.indices[t, j])
            y = wg[e] @ xx[t]
            rows.append(gate[t, j] * (wd[e] @ (torch.nn.functional.silu(y[:I]) * y[I:])))
        out = out + torch.stack(rows)
    (out * dout.double().cpu()).sum().backward()
    return out.detach().numpy(), [t.grad.numpy() for t in v]


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("T,E,k,H,I", [(1, 4, 2, 64, 32), (37, 6, 2, 128, 96), (90, 3, 3, 72, 40)])
def test_layer_forward_and_backward(lib, T, E, k, H, I, dt):
    """Route, group, both products, combine, and back: relative L2 against float64.  Roundings on the way, each at most
    half a step of its type: forward h, y (fp16), out; backward dy, dpre, dx and its sum, weights' gradients of rounded
    h and dpre.  Independent roundings add in L2 to at most the sum of their half steps: 4 of them in the 16-bit types
    at the outputs measured here (out: h, y, out; dx: pre, dy, dpre, dx, sum; the SwiGLU's curvature at most doubles
    what the rounded pre brings in)."""
    x, logits, gu, dn, dout = layer_case(T, T, E, k, H, I, dt)
    out, (dx, dl, dgu, ddn) = layer_reference(x, logits, gu, dn, k, dout)
    buf = q.moe_expert_layer_forward(x, logits, k, gu, dn, keep=True)
    g = q.moe_expert_layer_backward(dout, x, gu, dn, buf)
    rel = lambda got, ref: np.linalg.norm(f64(got) - ref) / np.linalg.norm(ref)  # noqa: E731
    step = HALF[dt]
    assert rel(buf.out, out) <= 2 * step + HALF["fp16"] + HALF["bf16"]
    assert g.dx.dtype == torch.bfloat16 and rel(g.dx, dx) <= 5 * step + HALF["bf16"]
    assert rel(g.ddown, ddn) <= 3 * step
    assert rel(g.dgate_up, dgu) <= 5 * step
    # by the logits: differences of dw between a token's slots, which cancel: against their magnitudes
    c = q.moe_unpermute_combine_grad(dout, buf.y_perm, buf.perm.pair_pos, buf.w, T, k, ids=buf.ids, E=E)
    amp = np.linalg.norm(f64(buf.w) * (np.linalg.norm(f64(dout), axis=1, keepdims=True)
                                       * np.sqrt(2.0) * np.sqrt((out ** 2).mean() * k * H)))
    assert np.linalg.norm(f64(g.dlogits) - dl) <= (2 * step + HALF["fp16"]) * amp
    assert torch.equal(c.dlogits, g.dlogits)
    if k == 1:
        assert (g.dlogits == 0).all()


def test_layer_backward_by_differences(lib):
    """Directional derivatives of <dout, layer(x, ...)> in float64 against the gradients."""
    T, E, k, H, I = 12, 4, 2, 64, 48
    x, logits, gu, dn, dout = layer_case(5, T, E, k, H, I, "fp16")
    buf = q.moe_expert_layer_forward(x, logits, k, gu, dn, keep=True)
    g = q.moe_expert_layer_backward(dout, x, gu, dn, buf)
    idn = buf.ids.long().cpu()
    v = [t.double().cpu() for t in (x, logits, gu, dn)]

    def loss(xx, lg, wg, wd):
        gate = torch.softmax(lg.gather(1, idn), -1)
        s = 0.0
        for t in range(T):
            for j in range(k):
                e = int(idn[t, j])
                y = wg[e] @ xx[t]
                s = s + gate[t, j] * (dout[t].double().cpu() @ (wd[e] @ (torch.nn.functional.silu(y[:I]) * y[I:])))
        return float(s)

    rng = np.random.default_rng(0)
    for i, grad in enumerate((g.dx, g.dlogits, g.dgate_up, g.ddown)):
        d = torch.from_numpy(rng.standard_normal(v[i].shape))
        h = 1e-4
        up = [t + h * d if j == i else t for j, t in enumerate(v)]
        dn_ = [t - h * d if j == i else t for j, t in enumerate(v)]
        want = (loss(*up) - loss(*dn_)) / (2 * h)
        got = float((grad.double().cpu() * d).sum())
        scale = float(grad.double().norm()) * 2  # a random direction's derivative is about the gradient's norm
        assert abs(got - want) <= (6 * HALF["fp16"] + HALF["bf16"]) * scale + 1e-3 * abs(want)


def test_layer_invalid_experts_add_nothing(lib):
    """Forward and backward with pairs whose id the grouping flagged (router ids replaced by hand)."""
    T, E, k, H, I = 9, 3, 2, 64, 32
    x, logits, gu, dn, dout = layer_case(6, T, E, k, H, I, "bf16")
    buf = q.alloc_expert_layer(T, E, k, H, I, DEV, keep=True)
    ids, w = q.moe_route_topk(logits, k)
    ids[3, 1], ids[7, :] = -1, 99
    p = q.moe_permute(ids, E)
    for name in ("counts", "seg_offsets", "sorted_pair", "pair_pos"):
        getattr(buf.perm, name).copy_(getattr(p, name))
    buf.ids.copy_(ids)
    buf.w.copy_(w)
    for t in (buf.pre, buf.h, buf.y_perm):
        t.fill_(float("nan"))  # what no call writes must not be read
    P, s = T * k, buf.perm.seg_offsets
    q.moe_grouped_gemm(gu, x, s, P, q.MOE_EPI_SWIGLU, gather_pair=buf.perm.sorted_pair, k=k, out=buf.h, pre=buf.pre)
    q.moe_grouped_gemm(dn, buf.h, s, P, q.MOE_EPI_NONE_F16, out=buf.y_perm)
    q.moe_unpermute_combine(buf.y_perm, buf.perm.pair_pos, buf.w, T, k, out=buf.out, n_valid=s[-1:])
    g = q.moe_expert_layer_backward(dout, x, gu, dn, buf)
    for t in (buf.out, g.dx, g.dlogits, g.dgate_up, g.ddown):
        assert torch.isfinite(t).all()
    assert (buf.out[7] == 0).all() and (g.dx[7] == 0).all() and (g.dlogits[7] == 0).all()


# --------------------------------------------------- streams, graphs, two at once
def test_layer_captured_and_replayed(lib):
    """A training step of the layer in one graph, replayed on new inputs between eager work, against eager calls."""
    T, E, k, H, I = 50, 8, 2, 128, 64
    x, logits, gu, dn, dout = layer_case(8, T, E, k, H, I, "bf16")
    buf = q.alloc_expert_layer(T, E, k, H, I, DEV, keep=True)

    def step():
        q.moe_expert_layer_forward(x, logits, k, gu, dn, buf=buf)
        return q.moe_expert_layer_backward(dout, x, gu, dn, buf)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = step()
    for i in range(4):
        new = layer_case(20 + i, T, E, k, H, I, "bf16")
        for dst, src in zip((x, logits, gu, dn, dout), new):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (buf.out, g.dx, g.dlogits, g.dgate_up, g.ddown)]
        b2 = q.moe_expert_layer_forward(*new[:2], k, *new[2:4], keep=True)
        e = q.moe_expert_layer_backward(new[4], new[0], new[2], new[3], b2)
        for a, b in zip(got, (b2.out, e.dx, e.dlogits, e.dgate_up, e.ddown)):
            assert torch.equal(a, b)


def test_two_streams_at_once(lib):
    """Two layers and two adapter additions on streams of their own, each given by `stream`."""
    cases = [layer_case(30 + i, 200, 8, 2, 256, 128, "bf16") for i in range(2)]
    want = []
    for x, logits, gu, dn, dout in cases:
        b = q.moe_expert_layer_forward(x, logits, 2, gu, dn, keep=True)
        want.append((b.out, *vars(q.moe_expert_layer_backward(dout, x, gu, dn, b)).values()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
        got = []
        for (x, logits, gu, dn, dout), s in zip(cases, streams):
            b = q.moe_expert_layer_forward(x, logits, 2, gu, dn, keep=True, stream=s)
            got.append((b.out, *vars(q.moe_expert_layer_backward(dout, x, gu, dn, b, stream=s)).values()))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for u, v in zip(a, b):
                assert torch.equal(u, v)


def test_adapters_on_another_stream_and_in_a_graph(lib):
    ids = [0] * 40 + [-1] * 3 + [1] * 2
    x, y, A, B, scale, p = adapter_batch(1, ids, 2, 16, 256, 320, "bf16", "bf16")
    want = q.moe_adapter_add(y, x, A, B, p.seg_offsets, p.sorted_pair, scale=scale)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = q.moe_adapter_add(y, x, A, B, p.seg_offsets, p.sorted_pair, scale=scale, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.moe_adapter_add(y, x, A, B, p.seg_offsets, p.sorted_pair, scale=scale, out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


# ------------------------------------------------ every path, beyond one tile each
@pytest.mark.parametrize("kernel", ["auto", "128", "256"])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_more_tiles_than_workgroups(lib, dt, kernel):
    """Workgroups go from tile to tile, the next one's loads under way (560 to 1360 tiles of 128): the ends of one
    tile and the starts of the next, an odd number of steps, segments and channels that end inside tiles."""
    kr = KERNELS[kernel]
    counts = [700, 0, 3, 130, 1200]
    for gather in (False, True):
        b = Batch(40, counts, 5128, 72, dt, k=2 if gather else 1, gather=gather)
        y, mag = do.product(f64(b.w), b.rows, b.offsets)
        args = dict(gather_pair=b.pairs, k=b.k, kernel=kr)
        close(f64(q.moe_grouped_gemm(b.w, b.a, b.seg, b.M, EPI[dt], **args)), y, bound(y, mag, 72, dt))
        pre = torch.empty(b.M, 5120, dtype=DT[dt], device=DEV)
        got = q.moe_grouped_gemm(b.w[:, :5120].contiguous(), b.a, b.seg, b.M, q.MOE_EPI_SWIGLU, pre=pre, **args)
        yy, mm = y[:, :5120], mag[:, :5120]
        close(f64(got), do.swiglu(yy), swiglu_bound(yy, mm, 72, dt), f"gather {gather}")
        close(f64(pre), yy, bound(yy, mm, 72, dt), f"pre gather {gather}")
        wide = Batch(41, counts, 520, 5128, dt, k=2 if gather else 1, gather=gather)
        dw, wmag = do.grad_weights(f64(wide.dy), wide.rows, wide.offsets)
        got = q.moe_grouped_gemm_grad_weights(wide.dy, wide.a, wide.seg, wide.E, wide.M, EPI[dt], gather_pair=wide.pairs,
                                              k=wide.k, kernel=kr)
        close(f64(got), dw, bound(dw, wmag, 1200, dt), f"gather {gather}")
    b = Batch(42, counts, 72, 5128, dt)
    da, mag = do.grad_rows(f64(b.w), f64(b.dy), b.offsets)
    close(f64(q.moe_grouped_gemm_grad_rows(b.w, b.dy, b.seg, b.M, q.MOE_EPI_NONE_F32, kernel=kr)), da, bound(da, mag, 72, "fp32"))
    p = dev(np.random.default_rng(1).standard_normal((b.M, 2 * 5128)), DT[dt])
    got = q.moe_grouped_gemm_grad_rows(b.w, b.dy, b.seg, b.M, q.MOE_EPI_SWIGLU_GRAD, pre=p, kernel=kr)
    close(f64(got), do.swiglu_grad(da, f64(p)), swiglu_grad_bound(da, 74 * 2.0 ** -23 * mag, f64(p), dt))


@pytest.mark.parametrize("counts", [[130, 150, 140, 129, 192, 137, 160, 131], [130, 150, 140, 129, 193, 137, 160, 131],
                                    [20, 300, 0, 15, 64, 65, 1, 128]])
def test_few_tiles(lib, counts):
    """Three stages: tiles of 128 rows, or of 256 where all segments have up to 192 and one round does."""
    for gather, K in ((False, 200), (True, 136)):
        b = Batch(43, counts, 4096, K, "bf16", k=2 if gather else 1, gather=gather)
        y, mag = do.product(f64(b.w), b.rows, b.offsets)
        for kr in (q.MOE_KERNEL_AUTO, q.MOE_KERNEL_TILE128):
            close(f64(q.moe_grouped_gemm(b.w, b.a, b.seg, b.M, gather_pair=b.pairs, k=b.k, kernel=kr)), y, bound(y, mag, K, "bf16"))
            got = q.moe_grouped_gemm(b.w, b.a, b.seg, b.M, q.MOE_EPI_SWIGLU, gather_pair=b.pairs, k=b.k, kernel=kr)
            close(f64(got), do.swiglu(y), swiglu_bound(y, mag, K, "bf16"))
    b = Batch(44, counts, 264, 4096, "fp16")
    da, mag = do.grad_rows(f64(b.w), f64(b.dy), b.offsets)
    pre = dev(np.random.default_rng(2).standard_normal((b.M, 2 * 4096)), torch.float16)
    for kr in (q.MOE_KERNEL_AUTO, q.MOE_KERNEL_TILE128):
        close(f64(q.moe_grouped_gemm_grad_rows(b.w, b.dy, b.seg, b.M, q.MOE_EPI_NONE_F16, kernel=kr)), da, bound(da, mag, 264, "fp16"))
        got = q.moe_grouped_gemm_grad_rows(b.w, b.dy, b.seg, b.M, q.MOE_EPI_SWIGLU_GRAD, pre=pre, kernel=kr)
        close(f64(got), do.swiglu_grad(da, f64(pre)), swiglu_grad_bound(da, 266 * 2.0 ** -23 * mag, f64(pre), "fp16"))


def test_offsets_and_pairs_outside_are_clamped(lib):
    """A table that runs past M_total, pairs past A's rows, an offset table that falls: rows stay inside the buffers."""
    b = Batch(45, [5, 5], 32, 24, "bf16")
    y, mag = do.product(f64(b.w), b.rows, b.offsets)
    for kr in KERNELS.values():
        far = i32([-7, 5, 1 << 30])
        close(f64(q.moe_grouped_gemm(b.w, b.a, far, 10, kernel=kr)), y, bound(y, mag, 24, "bf16"))
        close(f64(q.moe_grouped_gemm_grad_rows(b.w, b.dy, far, 10, q.MOE_EPI_NONE_F32, kernel=kr)),
              *(lambda r: (r[0], bound(r[0], r[1], 32, "fp32")))(do.grad_rows(f64(b.w), f64(b.dy), b.offsets)))
        dw, wmag = do.grad_weights(f64(b.dy), b.rows, b.offsets)
        close(f64(q.moe_grouped_gemm_grad_weights(b.dy, b.a, far, 2, 10, kernel=tile(kr))), dw, bound(dw, wmag, 5, "fp32"))
        out = torch.full((10, 32), 7.0, dtype=torch.bfloat16, device=DEV)
        q.moe_grouped_gemm(b.w, b.a, i32([6, 3, 9]), 10, out=out, kernel=kr)  # the first segment is empty
        assert (out[:3] == 7).all() and (out[9:] == 7).all() and not (out[3:9] == 7).all()
        pairs = i32([0, 1, 2, 3, 1 << 30, -5, 6, 7, 8, 9])
        got = f64(q.moe_grouped_gemm(b.w, b.a, b.seg, 10, gather_pair=pairs, kernel=kr))
        ok = [0, 1, 2, 3, 6, 7, 8, 9]
        close(got[ok], y[ok], bound(y, mag, 24, "bf16")[ok])


def test_the_same_row_many_times(lib):
    """Pairs of one token in many segments, and twice in one: the forward pass repeats it, the gradient counts it each time."""
    b = Batch(46, [40, 3, 90], 64, 72, "bf16", k=4, gather=True)
    pairs = np.concatenate([np.zeros(43, int), np.full(90, 5)])
    pairs[7] = 9
    rows = f64(b.a)[pairs // 4]
    y, mag = do.product(f64(b.w), rows, b.offsets)
    dw, wmag = do.grad_weights(f64(b.dy), rows, b.offsets)
    for kr in KERNELS.values():
        close(f64(q.moe_grouped_gemm(b.w, b.a, b.seg, b.M, gather_pair=i32(pairs), k=4, kernel=kr)), y, bound(y, mag, 72, "bf16"))
        close(f64(q.moe_grouped_gemm_grad_weights(b.dy, b.a, b.seg, b.E, b.M, gather_pair=i32(pairs), k=4, kernel=tile(kr))), dw,
              bound(dw, wmag, 90, "fp32"))


def test_combine_grad_of_a_repeated_expert(lib):
    """The same id in two slots of a token: both shares reach its logit."""
    ids = i32([[2, 2, 0]])
    p = q.moe_permute(ids, 3)
    y, dout = dev(np.random.default_rng(3).standard_normal((3, 16)), torch.float32), dev(np.ones((1, 16)), torch.bfloat16)
    w = dev([[0.5, 0.25, 0.25]], torch.float32)
    g = q.moe_unpermute_combine_grad(dout, y, p.pair_pos, w, 1, 3, ids=ids, E=3, n_valid=p.seg_offsets[-1:])
    dw, wn = f64(g.dw)[0], f64(w)[0]
    dl = wn * (dw - wn @ dw)
    close(f64(g.dlogits)[0], np.array([dl[2], 0, dl[0] + dl[1]]), 1e-5 * (1 + np.abs(dw).max()))


def test_two_graphs_with_one_workspace(lib):
    """Weights' gradients with split rows, captured twice with one workspace, replayed in turn between eager work."""
    cases = [Batch(50 + i, [2500, 700], 64, 40, "bf16") for i in range(2)]
    need = q.moe_grouped_gemm_grad_weights_workspace_size(2, 64, 40, 3200)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    want = [q.moe_grouped_gemm_grad_weights(b.dy, b.a, b.seg, 2, b.M) for b in cases]
    outs, graphs = [], []
    for b in cases:
        out = torch.empty(2, 64, 40, device=DEV)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            q.moe_grouped_gemm_grad_weights(b.dy, b.a, b.seg, 2, b.M, out=out, workspace=ws)
        outs.append(out)
        graphs.append(g)
    for _ in range(3):
        for out in outs:
            out.fill_(float("nan"))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        ws.fill_(255)
        for out, ref in zip(outs, want):
            assert torch.equal(out, ref)


def test_largest_batch_of_the_small_kernels(lib):
    """Row sums, lane sums and adapters over more slots and ranks than one pass takes (k = 300, rank 128, 1000 adapters)."""
    T, k, E, H = 2, 300, 1024, 2056
    r = np.random.default_rng(4)
    ids = np.stack([r.permutation(E)[:k] for _ in range(T)])
    p = q.moe_permute(i32(ids), E)
    y, dout = dev(r.standard_normal((T * k, H)), torch.float16), dev(r.standard_normal((T, H)), torch.bfloat16)
    w = torch.softmax(dev(r.standard_normal((T, k)), torch.float32), -1)
    g = q.moe_unpermute_combine_grad(dout, y, p.pair_pos, w, T, k, ids=i32(ids), E=E, n_valid=p.seg_offsets[-1:])
    dy, dw, mag, dl = do.combine_grad(f64(dout), f64(y), p.pair_pos.cpu().numpy().reshape(T, k), f64(w), T * k, ids, E)
    close(f64(g.dy), dy, (2.0 ** -8 + 2.0 ** -23) * np.abs(dy))
    close(f64(g.dw), dw, (H + 2) * 2.0 ** -23 * mag)
    e = (H + 2) * 2.0 ** -23 * mag.max()
    assert np.abs(f64(g.dlogits) - dl).max() <= f64(w).max() * 2 * (e + (k + 4) * 2.0 ** -23 * np.abs(dw).max())
    ids = r.integers(0, 1000, 300)
    x, y, A, B, scale, p = adapter_batch(6, ids.tolist(), 1000, 128, 40, 72, "bf16", "bf16")
    ref, mag = do.adapters(f64(y), f64(x), f64(A), f64(B), ids, f64(scale))
    got = q.moe_adapter_add(y, x, A, B, p.seg_offsets, p.sorted_pair, scale=scale)
    close(f64(got), ref, adapter_bound(ref, f64(y), mag, 40, 128, "bf16", "bf16"))


def test_most_tokens(lib):
    """2^24 - 1 tokens, of eight values each: the combine's gradient and an adapter, values that are exact."""
    T = (1 << 24) - 1
    t = torch.arange(T, dtype=torch.int32, device=DEV)
    v = (t % 251 - 125).to(torch.bfloat16)  # exact in bf16
    dout = v.view(T, 1).expand(T, 8).contiguous()
    p = q.Permutation(counts=None, seg_offsets=i32([0, T]), sorted_pair=t, pair_pos=t, workspace=None)
    g = q.moe_unpermute_combine_grad(dout, dout, p.pair_pos, torch.full((T, 1), 0.5, device=DEV), T, 1)
    assert torch.equal(g.dy, dout * 0.5) and torch.equal(g.dw.view(-1), 8 * v.float() ** 2)
    A, B = torch.ones(1, 8, 8, dtype=torch.bfloat16, device=DEV), torch.ones(1, 8, 8, dtype=torch.bfloat16, device=DEV)
    got = q.moe_adapter_add(dout, dout, A, B, p.seg_offsets, p.sorted_pair)
    assert torch.equal(got, (65 * v.float()).to(torch.bfloat16).view(T, 1).expand(T, 8))


def test_layer_of_no_tokens(lib):
    x, logits, gu, dn, dout = layer_case(9, 0, 4, 2, 64, 32, "bf16")
    buf = q.moe_expert_layer_forward(x, logits, 2, gu, dn, keep=True)
    g = q.moe_expert_layer_backward(dout, x, gu, dn, buf)
    assert buf.out.shape == g.dx.shape == (0, 64) and g.dlogits.shape == (0, 4)
    assert g.dgate_up.shape == gu.shape and (g.dgate_up == 0).all() and (g.ddown == 0).all()


README_CALLS = """buf = q.moe_expert_layer_forward(x, logits, k, gate_up, down, keep=True)        # [E][2I][H], [E][H][I]; buf.out bf16 [T][H]
grads = q.moe_expert_layer_backward(dout, x, gate_up, down, buf)                # .dx, .dlogits, .dgate_up, .ddown
p = q.moe_permute(adapter_ids, n)                                               # int32 [T][1]; -1: no adapter
q.moe_adapter_add(y, x, A, B, p.seg_offsets, p.sorted_pair, scale=scale, out=y)  # y[t] += scale[a] * B_a (A_a x[t])
"""


def test_calls_of_the_readme(lib):
    T, E, k, H, I, n, r = 20, 4, 2, 64, 32, 3, 8
    x, logits, gate_up, down, dout = layer_case(10, T, E, k, H, I, "bf16")
    ids = [t % 4 - 1 for t in range(T)]
    _, y, A, B, scale, _ = adapter_batch(3, ids, n, r, H, 40, "bf16", "bf16")
    names = dict(q=q, x=x, logits=logits, k=k, gate_up=gate_up, down=down, dout=dout, n=n, A=A, B=B, scale=scale, y=y.clone(),
                 adapter_ids=i32(ids).view(T, 1))
    exec(README_CALLS, names)
    (out, (dx, *_)) = layer_reference(x, logits, gate_up, down, k, dout)
    rel = lambda got, ref: np.linalg.norm(f64(got) - ref) / np.linalg.norm(ref)  # noqa: E731
    assert rel(names["buf"].out, out) <= 3 * HALF["bf16"] + HALF["fp16"] and rel(names["grads"].dx, dx) <= 6 * HALF["bf16"]
    ref, mag = do.adapters(f64(y), f64(x), f64(A), f64(B), ids, f64(scale))
    close(f64(names["y"]), ref, adapter_bound(ref, f64(y), mag, H, r, "bf16", "bf16"))
