"""Shared test setup: repo root on sys.path and the `gpu` marker.

Tests marked `gpu` need a real MI355X (gfx950) and the built HIP library; the
CPU suite (`-m "not gpu"`) covers the oracle against its pins, the synthetic
input generator, host-side logic of the boundary, and that the C-ABI library
loads and exports every symbol its header declares.
"""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


# Tests whose expected values are wrong, each with the proof; they run, and have to fail.
WRONG_VALUES = {
    "test_gpu_router.py::test_masked_and_extreme_logits":
        "takes p = exp(l - lse) with lse as it is returned, in fp32: of 70 logits of -1e30 each, lse = -1e30 + log 70 = -1e30, hence "
        "p = 1 for every expert, 70 in all, where p = 1/70 (and at 3e4, where lse is rounded by up to 2^-10, p is 5e-4 off); "
        "the same rows with their values: test_gpu_router_rows.py::test_gradient_of_masked_and_extreme_logits",
}


def pytest_collection_modifyitems(items):
    import pytest
    for item in items:
        for name, why in WRONG_VALUES.items():
            if f"/{item.nodeid}".split("[")[0].endswith(f"/{name}"):
                item.add_marker(pytest.mark.xfail(reason=why, raises=AssertionError, strict=True))


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X GPU and the built HIP library")
    config.addinivalue_line("markers", "slow: full-size workload (minutes of CPU oracle time)")
