"""The build: the C library needs nvcc alone, and the Python extension is of
the Python and torch that load it.  CPU only, with stand-ins for the
compilers."""
import os
import sys
import sysconfig

import pytest
import torch

from mla_latent_kv_dim_b200 import build as B

FAKE = """#!/bin/sh
# writes the file named after -o, or fails where $FAIL is set
[ -n "$FAIL" ] && { echo "no headers here" >&2; exit 1; }
while [ $# -gt 0 ]; do [ "$1" = -o ] && echo built > "$2"; shift; done
"""


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """Targets in a folder of their own, compilers that only write them."""
    for name in ("nvcc", "g++"):
        path = tmp_path / name
        path.write_text(FAKE)
        path.chmod(0o755)
    monkeypatch.setenv("NVCC", str(tmp_path / "nvcc"))
    monkeypatch.setenv("PATH", str(tmp_path) + os.pathsep + os.environ["PATH"])
    monkeypatch.setattr(B, "OBJ", str(tmp_path / "_build"))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "libtpla.so"))
    monkeypatch.setattr(B, "PKG", str(tmp_path))
    return tmp_path


def test_library_without_torch(tree, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)  # any import of it fails
    B.build(force=True)
    assert os.path.exists(B.LIB)


def test_library_without_a_cxx_compiler(tree, monkeypatch):
    """What the extension lacks is said by its own build, after the library's."""
    (tree / "g++").write_text("#!/bin/sh\nexit 1\n")
    B.build(force=True)
    assert os.path.exists(B.LIB)
    with pytest.raises(RuntimeError, match="compiler failed"):
        B.build_binding()


def test_command_line_builds_both_and_the_library_at_least(tree, monkeypatch, capsys):
    monkeypatch.setattr(sys, "argv", ["build"])
    assert B.main() == 0
    assert os.path.exists(B.LIB) and os.path.exists(B.binding_path())
    os.remove(B.binding_path())
    os.remove(B.LIB)
    (tree / "g++").write_text("#!/bin/sh\nexit 1\n")
    assert B.main() == 0
    assert os.path.exists(B.LIB) and not os.path.exists(B.binding_path())
    assert "kv_append" in capsys.readouterr().err


def test_extension_is_named_by_python_and_torch(tree, monkeypatch):
    path = B.binding_path()
    assert path.endswith(sysconfig.get_config_var("EXT_SUFFIX")) and torch.__version__ in path
    assert B.build_binding() == path and os.path.exists(path)
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    assert B.binding_path() != path
    other = B.build_binding()
    assert os.path.exists(other) and os.path.exists(path)


def test_extension_is_whole_or_absent(tree, monkeypatch):
    """A compiler that fails leaves no file that a later import would load."""
    monkeypatch.setenv("FAIL", "1")
    with pytest.raises(RuntimeError, match="no headers here"):
        B.build_binding()
    assert not os.path.exists(B.binding_path())
