import gc
import os
import sys
import time

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


def settle_readings(test, monkeypatch):
    """Where a test reads how much memory is allocated: nothing that tests before it left
    enters.  Garbage is collected and cached blocks given back first (a tensor that takes a cached
    block counts with the block's size, up to 1 MiB more than its own); and each reading
    waits for the work on the GPU and a moment more, as autograd's thread lets go of a pass's
    results only after the call that waited for them has returned."""
    if not {"memory_allocated", "max_memory_allocated"} & set(test.__code__.co_names):
        return
    import torch
    gc.collect()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    reading = torch.cuda.memory_allocated

    def settled(*args, **kwargs):
        torch.cuda.synchronize()
        time.sleep(0.02)
        return reading(*args, **kwargs)
    monkeypatch.setattr(torch.cuda, "memory_allocated", settled)


@pytest.fixture(autouse=True)
def _settled_readings(request, monkeypatch):
    if "gpu" in request.keywords:
        settle_readings(request.function, monkeypatch)
