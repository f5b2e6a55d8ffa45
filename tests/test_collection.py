"""What conftest.py keeps from running where it must not."""
import importlib.util
import pathlib
import types

import pytest
import torch

HERE = pathlib.Path(__file__).parent


def collected(file, name, marks=()):
    item = types.SimpleNamespace(path=HERE / file, originalname=name, keywords=set(marks), markers=[])
    item.add_marker = item.markers.append
    return item


@pytest.mark.parametrize("has_gpu", [False, True])
def test_made_up_addresses_never_meet_a_gpu(has_gpu, monkeypatch):
    spec = importlib.util.spec_from_file_location("conftest_under_test", HERE / "conftest.py")
    conftest = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(conftest)
    monkeypatch.setattr(torch.cuda, "is_available", lambda: has_gpu)
    fake = [collected("test_paged_abi.py", f"test_{x}_validation") for x in ("plan", "write", "attn", "select")]
    other = [collected("test_paged_abi.py", "test_workspace_sizes"), collected("test_abi.py", "test_validation")]
    gpu = [collected("test_paged_gpu.py", "test_attn", {"gpu"})]
    conftest.pytest_collection_modifyitems(None, fake + other + gpu)
    assert all(bool(i.markers) == has_gpu for i in fake)
    assert not any(i.markers for i in other)
    assert all(bool(i.markers) != has_gpu for i in gpu)
