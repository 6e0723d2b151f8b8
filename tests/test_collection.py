"""What conftest does for every test: which run where, on machines with and without a GPU, and
readings of allocated memory."""
import glob
import os
import threading
from pathlib import Path

import pytest

torch = pytest.importorskip("torch")
HERE = os.path.dirname(os.path.abspath(__file__))


class _Item:
    def __init__(self, name, gpu):
        self.path, self.keywords, self.skipped = Path(HERE) / name, {"gpu": 1} if gpu else {}, False

    def add_marker(self, mark):
        assert mark.name == "skip"
        self.skipped = True


def _collect(monkeypatch, have_gpu):
    import conftest
    monkeypatch.setattr(torch.cuda, "is_available", lambda: have_gpu)
    items = {n: _Item(n, gpu) for n, gpu in (("test_abi.py", False), ("test_attention_abi.py", False),
                                             ("test_around_abi.py", False), ("test_workloads.py", False), ("test_gpu_ffn.py", True))}
    conftest.pytest_collection_modifyitems(None, list(items.values()))
    return {n for n, it in items.items() if it.skipped}


def test_gpu_tests_are_skipped_without_a_gpu(monkeypatch):
    assert _collect(monkeypatch, False) == {"test_gpu_ffn.py"}


def test_calls_on_made_up_addresses_are_skipped_with_a_gpu(monkeypatch):
    assert _collect(monkeypatch, True) == {"test_abi.py", "test_attention_abi.py", "test_around_abi.py"}


def test_every_module_with_such_calls_is_named():
    """A call that only the missing device turns away has one of two statuses: no device, or
    another architecture."""
    import conftest
    found = set()
    for path in glob.glob(os.path.join(HERE, "test_*.py")):
        text = open(path).read()
        if "in (7" + ", 8)" in text and "mark.gpu" not in text:
            found.add(os.path.basename(path))
    assert found and found <= set(conftest.NEED_NO_GPU)


def test_readings_of_memory_wait_for_what_is_let_go_late(monkeypatch):
    """A stand-in for the allocator: a set of results that another thread lets go of a moment
    after the call that made it has returned, cached blocks and work behind."""
    import conftest
    done, held = [], [6]
    monkeypatch.setattr(torch.cuda, "synchronize", lambda: done.append("synchronize"))
    monkeypatch.setattr(torch.cuda, "empty_cache", lambda: done.append("empty_cache"))
    monkeypatch.setattr(torch.cuda, "memory_allocated", lambda: sum(held))

    def late():
        threading.Timer(0.002, held.clear).start()

    def reads():
        late()
        return torch.cuda.memory_allocated()

    def reads_nothing():
        return torch.cuda.synchronize

    with monkeypatch.context() as m:
        conftest.settle_readings(reads_nothing, m)
        assert not done and torch.cuda.memory_allocated() == 6
        conftest.settle_readings(reads, m)
        assert done == ["synchronize", "empty_cache"]
        assert reads() == 0
    held.append(6)
    assert torch.cuda.memory_allocated() == 6              # the reading itself is back
