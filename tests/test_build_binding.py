"""The compiled binding is rebuilt, and an old one refused, when the torch or the Python that it was compiled against changes;
the C library is built without torch."""
import os
import subprocess

import pytest

import sparse_bit_attention_smoothing_b200 as sg
from sparse_bit_attention_smoothing_b200 import build as sb


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A binding of its own in tmp_path, whose compiler only notes that it ran."""
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("module")
        return subprocess.CompletedProcess(cmd, 0, "", "")
    monkeypatch.setattr(sb, "LAYER_DIR", str(tmp_path))
    monkeypatch.setattr(sb.subprocess, "run", run)
    return ran


def versions(monkeypatch, torch_version):
    import importlib.metadata
    real = importlib.metadata.version
    monkeypatch.setattr(importlib.metadata, "version", lambda n: torch_version if n == "torch" else real(n))


def test_another_torch_rebuilds(tree, monkeypatch):
    first = sb.build_layer()
    assert os.path.exists(first) and len(tree) == 1
    assert sb.build_layer() == first and len(tree) == 1
    versions(monkeypatch, "9.9.9")
    second = sb.build_layer()
    assert second != first and len(tree) == 2 and os.listdir(sb.LAYER_DIR) == [os.path.basename(second)]
    assert sb.build_layer() == second and len(tree) == 2


def test_another_python_rebuilds(tree, monkeypatch):
    import sysconfig
    sb.build_layer()
    real = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var", lambda n: "cpython-399" if n == "SOABI" else real(n))
    sb.build_layer()
    assert len(tree) == 2


def test_other_flags_rebuild(tree, monkeypatch):
    sb.build_layer()
    monkeypatch.setattr(sb, "LAYER_FLAGS", sb.LAYER_FLAGS + ["-g"])
    sb.build_layer()
    assert len(tree) == 2 and "-g" in tree[1]


def test_a_binding_for_another_torch_is_not_loaded(monkeypatch):
    sb.build()
    monkeypatch.setattr(sg, "_layer_mod", None)
    assert sg._layer().__file__ == sb.layer_path()
    monkeypatch.setattr(sg, "_layer_mod", None)
    versions(monkeypatch, "9.9.9")
    with pytest.raises(RuntimeError, match="not built for this torch"):
        sg._layer()


def test_the_library_is_built_without_torch(tree, monkeypatch):
    import importlib.util
    real = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda n, *a: None if n == "torch" else real(n, *a))
    import builtins
    imp = builtins.__import__

    def no_torch(name, *a, **kw):
        if name.split(".")[0] == "torch":
            raise ModuleNotFoundError("No module named 'torch'", name="torch")
        return imp(name, *a, **kw)
    monkeypatch.setattr(builtins, "__import__", no_torch)
    assert sb.build() == sb.LIB and os.path.exists(sb.LIB)
    assert not any("binding.cpp" in " ".join(c) for c in tree)
