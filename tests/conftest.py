import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (GB300, sm_103a)")
    config.addinivalue_line("markers", "slow: long-running CPU test")


# Tests of the host side that make allowed calls on addresses that are none, which end at
# "no device" on a machine without a GPU and would be read by kernels on one.
HOST_ONLY = {"tests/test_experts_cpu.py::" + name
             for name in ("test_sort_sizes", "test_gather_sizes", "test_combine_sizes",
                          "test_combine_backward_sizes")}


def pytest_collection_modifyitems(config, items):
    try:
        import torch
        have_gpu = torch.cuda.is_available()
    except Exception:  # pragma: no cover
        have_gpu = False
    if have_gpu:
        skip = pytest.mark.skip(reason="calls on addresses that are none: for machines without a GPU")
        for item in items:
            if "tests/" + item.nodeid.split("tests/")[-1] in HOST_ONLY:
                item.add_marker(skip)
        return
    skip = pytest.mark.skip(reason="no CUDA GPU in this process")
    for item in items:
        if "gpu" in item.keywords:
            item.add_marker(skip)
