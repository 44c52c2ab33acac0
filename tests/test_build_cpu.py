"""When the marshalling of the draft-tree calls is built anew."""
import importlib.util
import types

import pytest

from gated_delta_rule_27_gb300 import build


@pytest.fixture
def compiled(tmp_path, monkeypatch):
    """build_tree_py with a compiler that only writes its output down, and a torch whose version can be changed."""
    runs = []

    def run(cmd, **_):
        runs.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    torch = tmp_path / "torch"
    torch.mkdir()
    (torch / "version.py").write_text("__version__ = '1'")
    monkeypatch.setattr(build, "TREE_PY", str(tmp_path / "_kda_tree.so"))
    monkeypatch.setattr(build, "TREE_PY_FOR", str(tmp_path / "_kda_tree.txt"), raising=False)
    monkeypatch.setattr(build.subprocess, "run", run)
    monkeypatch.setattr(importlib.util, "find_spec", lambda name: types.SimpleNamespace(submodule_search_locations=[str(torch)]))
    return runs, torch


def test_another_torch_makes_the_marshalling_stale(compiled):
    runs, torch = compiled
    build.build_tree_py()
    assert len(runs) == 1
    build.build_tree_py()
    assert len(runs) == 1  # fresh
    (torch / "version.py").write_text("__version__ = '2'")
    build.build_tree_py()
    assert len(runs) == 2
    build.build_tree_py()
    assert len(runs) == 2
