"""Host tests that pass made-up pointers through every check of the host are skipped where a GPU is
present, whatever else the run selects."""
import importlib

import pytest

from tests import conftest as G


class Item:
    def __init__(self, file, name):
        self.fspath, self.name, self.marks = f"/somewhere/tests/{file}", name, []

    def add_marker(self, m):
        self.marks.append(m.name)


@pytest.mark.parametrize("present", [False, True])
def test_made_up_pointers_stay_off_a_gpu(monkeypatch, present):
    monkeypatch.setattr(G, "gpu_present", lambda: present)
    named = [Item(f, n) for f, names in G.MADE_UP_POINTERS.items() for n in names]
    other = [Item("test_zz_no_alloc.py", "test_noalloc_matches_forward_on_consecutive_calls"),
             Item("test_other.py", "test_noalloc_size_limit")]
    G.pytest_collection_modifyitems(named + other)
    assert len(named) == 3
    assert all(i.marks == (["skip"] if present else []) for i in named)
    assert not any(i.marks for i in other)


def test_the_named_tests_are_there():
    for f, names in G.MADE_UP_POINTERS.items():
        m = importlib.import_module("tests." + f[:-3])
        assert all(callable(getattr(m, n)) for n in names)
