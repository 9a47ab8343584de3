"""Tests of argument checks whose good calls would launch on addresses that are none stay away from a GPU (CPU)."""
import os
import types

import pytest

from tests import conftest


class Item:
    def __init__(self, path, name):
        self.fspath, self.originalname, self.markers = path, name, []

    def add_marker(self, m):
        self.markers.append(m.name)


@pytest.mark.parametrize("available, expr, skipped", [(True, "", True), (False, "", False), (True, "gpu", False),
                                                      (True, "not gpu", False)])
def test_they_are_left_out_beside_a_gpu(monkeypatch, available, expr, skipped):
    import torch
    monkeypatch.setattr(torch.cuda, "is_available", lambda: available)
    monkeypatch.setenv("CUDA_VISIBLE_DEVICES", "0")
    config = types.SimpleNamespace(option=types.SimpleNamespace(markexpr=expr), addinivalue_line=lambda *a: None)
    conftest.pytest_configure(config)
    assert os.environ["CUDA_VISIBLE_DEVICES"] == ("" if expr == "not gpu" else "0")
    names = ("test_null_and_misaligned_pointers", "test_no_tokens_need_no_rows", "test_append_arguments")
    items = [Item("tests/test_rope_abi.py", n) for n in names]
    other = [Item("tests/test_zz_no_alloc.py", "test_x"), Item("tests/test_rope_abi.py", "test_bad_problems"),
             Item("tests/test_cache_abi.py", names[0])]
    every = [*other, *items]
    conftest.pytest_collection_modifyitems(config, every)
    assert [i.markers for i in items] == [["skip"] if skipped else []] * 3 and not any(i.markers for i in other)
    assert every[-1] is other[0]        # the last file stays the last
