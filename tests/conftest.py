import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a) and the built extension")


def pytest_collection_modifyitems(config, items):
    try:
        import torch
        has_gpu = torch.cuda.is_available()
    except Exception:  # pragma: no cover
        has_gpu = False
    if has_gpu:
        # Calls on made-up device addresses.  Some are refused for want of a workspace, which the same
        # sizes do not need on a real GPU: there they would be launched and fault.
        skip = pytest.mark.skip(reason="made-up device addresses: run where there is no GPU")
        for item in items:
            if item.path.name == "test_paged_abi.py" and getattr(item, "originalname", "").endswith("_validation"):
                item.add_marker(skip)
        return
    skip = pytest.mark.skip(reason="no CUDA device")
    for item in items:
        if "gpu" in item.keywords:
            item.add_marker(skip)
