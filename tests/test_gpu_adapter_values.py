"""GPU checks of what the adapters' first product v = A_a x may be: any fp32
number, whatever the operands' type, beside the values near 1 that other tests
use.  Against float64.

Tolerances.  A sum of n products that are exact in fp32 is off by at most
n * 2^-23 times the sum of their magnitudes (an addition cut, not rounded).
The second product multiplies v as three bf16 numbers, exactly, by B's one
(bf16) or two (fp16): up to 6 r products; scale, addition and the output's
rounding add a few roundings.  Where every sum has an exact fp32 value, the
result has to be that value.
"""
import numpy as np
import pytest
import torch

import quantized_moe_expert_top_amd as q

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}


def f64(t):
    return t.double().cpu().numpy()


def dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV).to(dtype)


def group(ids, n):
    return q.moe_permute(torch.tensor(ids, dtype=torch.int32, device=DEV).view(-1, 1), n)


def reference(y, x, A, B, ids, scale):
    """float64, and the magnitudes behind each sum."""
    out, mag = f64(y), np.zeros(tuple(y.shape))
    ids, xs = np.asarray(ids), f64(x)
    for a in np.unique(ids):
        if 0 <= a < A.shape[0]:
            t, Aa, Ba = ids == a, f64(A[a]), f64(B[a])
            out[t] += scale[a] * (xs[t] @ Aa.T @ Ba.T)
            mag[t] = abs(scale[a]) * (np.abs(xs[t]) @ np.abs(Aa).T @ np.abs(Ba).T)
    return out, mag


def bound(ref, mag, K, r, y_dt):
    """Both sums, three roundings (the scale's, the addition's and the reference's own), the output's."""
    tiny = 2.0 ** -25 if y_dt == "fp16" else 0.0
    return HALF[y_dt] * np.abs(ref) * (1 + 2.0 ** -20) + tiny + mag * (K + 6 * r + 8) * 2.0 ** -23


def close(got, ref, tol):
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} off, first at {np.argwhere(bad)[0]}: {got[bad][0]} for " \
        f"{ref[bad][0]} (tolerance {np.broadcast_to(tol, ref.shape)[bad][0]})"


@pytest.mark.parametrize("r,N", [(8, 40), (32, 72), (40, 136), (128, 264)])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_every_bit_of_the_first_product(lib, dt, r, N):
    """v of 24 bits, channel c reads rank c % r alone by a power of two: out is v times that, to the last bit."""
    g = np.random.default_rng(r)
    T, K = 37, 16
    x, A, B = np.zeros((T, K)), np.zeros((1, r, K)), np.zeros((1, N, r))
    x[:, :3] = np.array([1, 2.0 ** -8, 2.0 ** -16]) * 2.0 ** g.integers(-4, 5, (T, 1))
    A[0, :, :3] = g.integers(128, 256, (r, 3)) * g.choice([-1, 1], (r, 1))  # one sign: 24 bits in a row
    c = np.arange(N)
    B[0, c, c % r] = 2.0 ** g.integers(-3, 4, N)
    x, A, B, y = dev(x, DT[dt]), dev(A, DT[dt]), dev(B, DT[dt]), torch.zeros(T, N, device=DEV)
    p = group([0] * T, 1)
    want = f64(x) @ f64(A[0]).T @ f64(B[0]).T
    assert np.array_equal(want, want.astype(np.float32))
    assert np.array_equal(f64(q.moe_adapter_add(y, x, A, B, p.seg_offsets, p.sorted_pair)), want)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_first_products_of_every_size_in_one_token(lib, dt):
    """Ranks from 2^-30 to 2^17 beside each other in one token, each read by channels of its own, and by all at once."""
    g = np.random.default_rng(3)
    T, K, r, N = 20, 64, 48, 200
    size = 2.0 ** np.arange(-30, 18)
    x = g.standard_normal((T, K))
    A = g.standard_normal((1, r, K)) * np.minimum(size, 2.0 ** 8)[:, None] / 8
    # fp16's own range ends at 2^-24: the smallest and the largest come from x's channels, not from A
    x[:, :8], x[:, 8:16] = x[:, :8] * 2.0 ** -10, x[:, 8:16] * 2.0 ** 9
    A[0, :18] = np.concatenate([g.standard_normal((18, 8)) * size[:18, None] * 2.0 ** 10, np.zeros((18, K - 8))], 1)
    A[0, 38:] = np.concatenate([np.zeros((10, 8)), g.standard_normal((10, 8)) * size[38:, None] * 2.0 ** -9,
                                np.zeros((10, K - 16))], 1)
    B = np.zeros((1, N, r))
    c = np.arange(N - 8)
    B[0, c, c % r] = g.standard_normal(N - 8)
    B[0, N - 8:] = g.standard_normal((8, r))
    x, A, B, y = dev(x, DT[dt]), dev(A, DT[dt]), dev(B, DT[dt]), torch.zeros(T, N, device=DEV)
    p = group([0] * T, 1)
    ref, mag = reference(y, x, A, B, [0] * T, [1.0])
    close(f64(q.moe_adapter_add(y, x, A, B, p.seg_offsets, p.sorted_pair)), ref, bound(ref, mag, K, r, "fp32"))


@pytest.mark.parametrize("y_dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("r,small", [(8, 12), (16, 20), (64, 24), (128, 20)])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_small_first_products_with_a_large_scale(lib, dt, r, small, y_dt):
    """A and x of 2^-(small / 2) each, a scale that brings the product back."""
    g = np.random.default_rng(small)
    T, K, N = 45, 72, 136
    ids = [t % 3 - 1 for t in range(T)]
    x, A = g.standard_normal((T, K)) * 2.0 ** -(small / 2), g.standard_normal((2, r, K)) * 2.0 ** -(small / 2)
    x, A, B = dev(x, DT[dt]), dev(A, DT[dt]), dev(g.standard_normal((2, N, r)) / 64, DT[dt])
    y = dev(g.standard_normal((T, N)) / 1024, DT[y_dt])
    scale = dev([2.0 ** small, -(2.0 ** small) / 3], torch.float32)
    p = group(ids, 2)
    ref, mag = reference(y, x, A, B, ids, f64(scale))
    close(f64(q.moe_adapter_add(y, x, A, B, p.seg_offsets, p.sorted_pair, scale=scale)), ref, bound(ref, mag, K, r, y_dt))


@pytest.mark.parametrize("r", [8, 24, 64, 128])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_large_first_products(lib, dt, r):
    """v past 65504, fp16's largest number, and up to 10^8: finite, as the sums are."""
    g = np.random.default_rng(r)
    T, K, N = 33, 40, 72
    x, A = dev(g.standard_normal((T, K)) * 1000, DT[dt]), dev(g.standard_normal((1, r, K)) * 1000, DT[dt])
    B, y = dev(g.standard_normal((1, N, r)), DT[dt]), dev(g.standard_normal((T, N)), torch.float32)
    scale, p = dev([2.0 ** -20], torch.float32), group([0] * T, 1)
    ref, mag = reference(y, x, A, B, [0] * T, f64(scale))
    close(f64(q.moe_adapter_add(y, x, A, B, p.seg_offsets, p.sorted_pair, scale=scale)), ref, bound(ref, mag, K, r, "fp32"))
    x, A, B = dev(np.full((2, 16), 60000.0), DT[dt]), dev(np.ones((1, r, 16)), DT[dt]), dev(np.ones((1, 40, r)), DT[dt])
    p = group([0, 0], 1)
    got = q.moe_adapter_add(torch.ones(2, 40, device=DEV), x, A, B, p.seg_offsets, p.sorted_pair)
    assert (got == 1 + r * 16 * float(x[0, 0])).all()


@pytest.mark.parametrize("r", [8, 16, 32, 40, 128])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_infinite_entries_of_the_second_factor(lib, dt, r):
    """An infinite entry of B makes its channels infinite, with the sign of its product by v; by v = 0 not a number."""
    T, K, N = 18, 16, 72
    x, A, B = np.zeros((T, K)), np.zeros((1, r, K)), np.ones((1, N, r))
    x[:, 0] = np.resize([1, 0.5, 3, 1.5, 2.0 ** -14, -1], T)  # v as one, two and three bf16 numbers
    x[:, 1] = np.resize([0, 2.0 ** -9, 0], T)
    x[:, 2] = 2.0 ** -14
    A[0, :, 0] = A[0, :, 1] = 1
    A[0, : r // 2, 2] = 2.0 ** -8
    A[0, r - 1] = 0  # v = 0
    B[0, 3, 0], B[0, 4, 1], B[0, 9, 2], B[0, 9, 3] = np.inf, -np.inf, np.inf, np.inf
    B[0, 20, 0], B[0, 20, 1], B[0, 30, r - 1], B[0, 40, 2] = np.inf, -np.inf, np.inf, np.nan
    x, A, B, y = dev(x, DT[dt]), dev(A, DT[dt]), dev(B, DT[dt]), torch.ones(T, N, device=DEV)
    p = group([0] * T, 1)
    got = f64(q.moe_adapter_add(y, x, A, B, p.seg_offsets, p.sorted_pair))
    with np.errstate(invalid="ignore"):
        v = f64(x) @ f64(A[0]).T
        want = 1 + (v[:, None, :] * f64(B[0])[None]).sum(-1)
    odd = [3, 4, 9, 20, 30, 40]
    assert np.array_equal(got[:, odd], want[:, odd], equal_nan=True)
    assert np.isinf(want[:, [3, 4, 9]]).all() and np.isnan(want[:, [20, 30, 40]]).all()
    rest = np.setdiff1d(np.arange(N), odd)
    assert np.isfinite(want[:, rest]).all()
    close(got[:, rest], want[:, rest], (1 + (K + 6 * r + 8) * np.abs(v).sum(1, keepdims=True)) * 2.0 ** -23)


@pytest.mark.parametrize("r", [16, 32, 64, 128])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_first_products_that_are_not_finite(lib, dt, r):
    """+-infinite and NaN first products beside finite ones: what the sums give."""
    T, K, N = 6, 16, 40
    x, A, B = np.ones((T, K)), np.zeros((1, r, K)), np.ones((1, N, r))
    A[0, :, 0], A[0, 0, 1], A[0, 1, 2] = 1, 1, 1
    x[0, 1], x[1, 1], x[2, 1], x[2, 2], x[3, 2] = np.inf, -np.inf, np.inf, -np.inf, np.nan
    A[0, 1:, 1], A[0, 0, 2], A[0, 2:, 2] = 0, 0, 0
    B[0, 5] = -2
    x, A, B, y = dev(x, DT[dt]), dev(A, DT[dt]), dev(B, DT[dt]), torch.ones(T, N, device=DEV)
    p = group([0] * T, 1)
    got = f64(q.moe_adapter_add(y, x, A, B, p.seg_offsets, p.sorted_pair))
    with np.errstate(invalid="ignore"):
        want = 1 + (f64(x) @ f64(A[0]).T) @ f64(B[0]).T
    assert np.isnan(want[:4]).all()  # infinite inputs meet A's zeros in the other ranks
    assert np.array_equal(got, want, equal_nan=True)
    x[:4] = 1
    A[0, :, 3] = 3.0e38 if dt == "bf16" else 6.0e4
    x[0, 3], x[1, 3] = float("inf"), -float("inf")
    got = f64(q.moe_adapter_add(y, x, A, B, p.seg_offsets, p.sorted_pair))
    assert (got[0, 5], got[1, 5]) == (-np.inf, np.inf) and (np.delete(got[0], 5) == np.inf).all() and (np.delete(got[1], 5) == -np.inf).all()


# chunks of 64 channels that a wavefront of the kernel goes through: N / 64 over 8 wavefronts (ranks above 64: 4), when
# the tokens' tiles, one per adapter at least, fill the chip without a split of the channels
MANY = [0] * 70 + [1] * 33 + [-1] * 5 + list(range(3, 262)) + [2] * 16 + [300]


@pytest.mark.parametrize("r,N", [(r, N) for r in (8, 32, 40) for N in (520, 1032, 1544, 2056, 2600, 3592)]
                         + [(128, N) for N in (264, 520, 776, 1032, 1800)])
@pytest.mark.parametrize("dt,y_dt", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp32"), ("fp16", "fp32")])
def test_many_chunks_of_channels(lib, dt, y_dt, r, N):
    """Two to eight chunks per wavefront, the next ones under way, also in place."""
    g = torch.Generator(device=DEV).manual_seed(r * N)
    K, n, T = 24, 262, len(MANY)
    mk = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x, y, A, B = mk(T, K).to(DT[dt]), mk(T, N).to(DT[y_dt]), (mk(n, r, K) / 5).to(DT[dt]), mk(n, N, r).to(DT[dt])
    scale = 0.5 + torch.rand(n, generator=g, device=DEV)
    p = group(MANY, n)
    ref, mag = reference(y, x, A, B, MANY, f64(scale))
    got = q.moe_adapter_add(y, x, A, B, p.seg_offsets, p.sorted_pair, scale=scale)
    close(f64(got), ref, bound(ref, mag, K, r, y_dt))
    bare = [t for t, a in enumerate(MANY) if not 0 <= a < n]
    assert torch.equal(got[bare], y[bare])
    into = y.clone()
    assert q.moe_adapter_add(into, x, A, B, p.seg_offsets, p.sorted_pair, scale=scale, out=into) is into
    assert torch.equal(into, got)


@pytest.mark.parametrize("r", [8, 32, 64, 128])
@pytest.mark.parametrize("exponent", [60, 98])
def test_first_products_near_the_least(lib, r, exponent):
    """bf16: v of 2^-60 and 2^-98, brought back by the scale."""
    g = np.random.default_rng(exponent + r)
    T, K, N = 21, 40, 72
    x, A = g.standard_normal((T, K)) * 2.0 ** -(exponent // 2), g.standard_normal((1, r, K)) * 2.0 ** -(exponent // 2)
    x, A, B = dev(x, DT["bf16"]), dev(A, DT["bf16"]), dev(g.standard_normal((1, N, r)), DT["bf16"])
    y, scale, p = torch.zeros(T, N, device=DEV), dev([2.0 ** exponent], torch.float32), group([0] * T, 1)
    ref, mag = reference(y, x, A, B, [0] * T, f64(scale))
    close(f64(q.moe_adapter_add(y, x, A, B, p.seg_offsets, p.sorted_pair, scale=scale)), ref, bound(ref, mag, K, r, "fp32"))
