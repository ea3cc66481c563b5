"""Which parts of the build need what."""
import importlib.util
import os
import subprocess
import sysconfig
import types

import pytest

from decoder_only_transformer_fwd_b200 import build


@pytest.mark.parametrize("missing", ["torch", "headers"])
def test_the_c_library_builds_without_torch_or_python_headers(missing, monkeypatch, tmp_path, capsys):
    """libnc.so needs nvcc alone; the Python binding's native part is left out, and said to be."""
    monkeypatch.setattr(build, "PYLIB", str(tmp_path / "_ncpy.so"))
    if missing == "torch":
        find = importlib.util.find_spec
        monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    else:
        paths = dict(sysconfig.get_paths(), include=str(tmp_path))
        monkeypatch.setattr(sysconfig, "get_paths", lambda *a, **k: paths)
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert not os.path.exists(build.PYLIB)
    assert "_ncpy.so" in capsys.readouterr().err


def test_the_binding_is_built_again_for_another_torch_or_python(monkeypatch, tmp_path):
    """An upgrade of either leaves the sources as they are, and the old file does not load any more."""
    calls = []

    def compiler(cmd, **kw):
        calls.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return subprocess.CompletedProcess(cmd, 0, "", "")

    torch_dir = tmp_path / "torch"
    torch_dir.mkdir()
    (torch_dir / "version.py").write_text("__version__ = '1'\n")
    monkeypatch.setattr(build, "PYLIB", str(tmp_path / "_ncpy.so"))
    monkeypatch.setattr(build, "OBJ", str(tmp_path))
    monkeypatch.setattr(subprocess, "run", compiler)
    monkeypatch.setattr(importlib.util, "find_spec", lambda name: types.SimpleNamespace(submodule_search_locations=[str(torch_dir)]))
    for want in (1, 1):                                      # the second time it is up to date
        assert build.build_py() == build.PYLIB and len(calls) == want
    (torch_dir / "version.py").write_text("__version__ = '2'\n")
    for want in (2, 2):
        assert build.build_py() == build.PYLIB and len(calls) == want
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: ".another-python.so")
    for want in (3, 3):
        assert build.build_py() == build.PYLIB and len(calls) == want
