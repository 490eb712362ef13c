"""What pytest leaves out on machines with and without a GPU."""
import pytest
import torch

from tests import conftest


class _Item:
    def __init__(self, nodeid, *keywords):
        self.nodeid, self.keywords, self.marks = nodeid, keywords, []

    def add_marker(self, mark):
        self.marks.append(mark.name)


@pytest.mark.parametrize("root", ["tests/", "", "repo/tests/"])
def test_calls_on_fake_addresses_stay_off_the_gpu(monkeypatch, root):
    """The allowed calls of test_experts_cpu.py, on the address 256, run no kernel anywhere."""
    names = ["test_sort_sizes", "test_gather_sizes", "test_combine_sizes",
             "test_combine_backward_sizes"]
    for gpu in (False, True):
        monkeypatch.setattr(torch.cuda, "is_available", lambda: gpu)
        fake = [_Item(f"{root}test_experts_cpu.py::{n}") for n in names]
        other = _Item(f"{root}test_experts_cpu.py::test_sort_refuses[bad0]")
        on_gpu = _Item(f"{root}test_experts_gpu.py::test_refusals", "gpu")
        conftest.pytest_collection_modifyitems(None, [*fake, other, on_gpu])
        assert all(i.marks == (["skip"] if gpu else []) for i in fake)
        assert other.marks == [] and on_gpu.marks == ([] if gpu else ["skip"])
