import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a) and the built library")
    config.addinivalue_line("markers", "no_device: hands made-up addresses to calls that only a missing GPU stops")


# Tests that carry no mark and do the same as those marked no_device: valid calls with made-up
# addresses, which end at device discovery.  Where there is a GPU the kernels would read those addresses.
MADE_UP_ADDRESSES = {"test_score_plan_fits_every_supported_shape", "test_an_empty_list_tensor_is_no_error",
                     "test_a_workspace_serves_smaller_calls"}


def gpu_available() -> bool:
    try:
        import torch
        return torch.cuda.is_available()
    except Exception:
        return False


def pytest_collection_modifyitems(config, items):
    if gpu_available():
        skip = pytest.mark.skip(reason="made-up addresses: not where there is a GPU")
        for item in items:
            if "no_device" in item.keywords or getattr(item, "originalname", None) in MADE_UP_ADDRESSES:
                item.add_marker(skip)
        return
    skip = pytest.mark.skip(reason="no CUDA device")
    for item in items:
        if "gpu" in item.keywords:
            item.add_marker(skip)
