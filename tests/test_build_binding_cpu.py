"""The binding's extension goes with one PyTorch: another version, or an extension of unknown origin, is built again, and
one that was not is refused."""
import os
import types

import pytest

from fp4_compressed_sparse_kv_b200 import build, csa


def test_built_again_for_another_torch(tmp_path, monkeypatch):
    so, stamp = tmp_path / "_runs.so", tmp_path / "_runs.stamp"
    monkeypatch.setattr(build, "RUNS", str(so))
    monkeypatch.setattr(build, "RUNS_STAMP", str(stamp), raising=False)
    compiled = []

    def run(cmd, **kw):
        compiled.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(build.subprocess, "run", run)
    so.write_text("newer than its sources, of an unknown PyTorch")
    build._build_binding()
    assert len(compiled) == 1
    build._build_binding()
    assert len(compiled) == 1                     # up to date
    import importlib.metadata
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "99.0")
    build._build_binding()
    assert len(compiled) == 2 and os.path.exists(so)
    build._build_binding()
    assert len(compiled) == 2


def test_refused_under_another_torch(monkeypatch):
    build.build()
    monkeypatch.setattr(csa, "_runs_mod", None)
    monkeypatch.setattr(csa.torch, "__version__", "99.0+cu1")
    with pytest.raises(ImportError, match="99.0"):
        csa._runs()
    monkeypatch.undo()
    assert csa._runs() is not None
