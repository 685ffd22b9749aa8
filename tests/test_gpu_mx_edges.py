"""GPU checks of the MX operators at the ends of their ranges, against the
float64 references (oracle/mx_oracle.py).

Tolerances are those of test_gpu_mx.py.
"""
import numpy as np
import pytest

from tests.test_gpu_mx import check_route

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
