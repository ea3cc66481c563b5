"""Which parts of the build need what."""
import importlib.util
import os
import sysconfig

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
