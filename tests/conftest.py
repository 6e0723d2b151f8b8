import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")


# These call entry points with arguments that are valid in every way, at addresses made up:
# nothing but the missing device keeps the library from launching kernels on them.
NEED_NO_GPU = ("test_abi.py", "test_attention_abi.py", "test_around_abi.py")


def pytest_collection_modifyitems(config, items):
    # GPU tests are skipped (not failed) where no GPU is visible; on a machine with a GPU
    # they run and must find the built library, and what needs a machine without one is skipped.
    try:
        import torch
        have_gpu = torch.cuda.is_available()
    except Exception:  # pragma: no cover
        have_gpu = False
    skip = pytest.mark.skip(reason="its calls would launch on made-up addresses" if have_gpu else "no GPU visible")
    for it in items:
        if it.path.name in NEED_NO_GPU if have_gpu else "gpu" in it.keywords:
            it.add_marker(skip)
