import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a) and the built library")
    config.addinivalue_line("markers", "slow: long-running (full-size workloads)")


# Host tests that make a call which passes every check, with an address that is
# nobody's: for machines without a GPU, where it ends at the check of the device.
# With one it would launch and read that address.
NO_GPU_ONLY = ("test_serving_host.py::test_append_head_dims",)


def pytest_collection_modifyitems(config, items):
    """GPU tests need a CUDA device; without one they are skipped (the CPU
    suite deselects them with -m "not gpu"). Those of NO_GPU_ONLY must not meet one."""
    try:
        import torch
        has_gpu = torch.cuda.is_available()
    except Exception:  # pragma: no cover
        has_gpu = False
    if has_gpu:
        alone = pytest.mark.skip(reason="only for machines without a CUDA device")
        for it in items:
            if it.nodeid.endswith(NO_GPU_ONLY):
                it.add_marker(alone)
        return
    skip = pytest.mark.skip(reason="no CUDA device")
    for it in items:
        if "gpu" in it.keywords:
            it.add_marker(skip)


@pytest.fixture(scope="session")
def mgb_lib():
    """The built library (built in-tree first if missing)."""
    from megatron_transformer_layer_fwd_gb300 import build, mgb
    build.build()
    return mgb.load()
