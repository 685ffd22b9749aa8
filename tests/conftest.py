import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")


# Tests whose expected value is wrong, each with the proof; a right library fails them.
WRONG_VALUES = {
    "tests/test_gpu_dense.py::test_adapters_past_the_range[fp16]":
        "its last line expects infinity where A x is 16 * 60000 = 960000: finite in fp32, which A x is held in, and "
        "1 + r * 960000 (r = 8: 7680001, exact; r = 24: 23040001, rounded to fp32) is the result; "
        "tests/test_gpu_adapter_values.py::test_large_first_products holds the right value, and "
        "test_first_products_that_are_not_finite the infinite rows",
}


def pytest_collection_modifyitems(items):
    for item in items:
        if item.nodeid in WRONG_VALUES:
            item.add_marker(pytest.mark.xfail(reason=WRONG_VALUES[item.nodeid], raises=AssertionError, strict=True))


def gpu_available() -> bool:
    try:
        import torch
        return torch.cuda.is_available()
    except Exception:
        return False


@pytest.fixture(scope="session")
def lib():
    """The HIP library through its Python binding (GPU tests only)."""
    if not gpu_available():
        pytest.skip("no GPU")
    import quantized_moe_expert_top_amd as q
    return q
