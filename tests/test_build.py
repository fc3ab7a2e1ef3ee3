"""build(): the library takes nvcc alone; the host-side binding is made beside it where
PyTorch, g++ and Python's headers are there.  Both compilers are stand-ins here."""
import glob
import os
import subprocess
import sys
import sysconfig

import pytest

import speculative_decoding_verify_03_gb300 as m

GXX = """#!/bin/sh
while [ "$1" != -o ]; do shift; done
echo made > "$2"
exit {code}
"""


@pytest.fixture
def tree(monkeypatch, tmp_path):
    """A place for what is built, a g++ that writes its output and says `code`."""
    monkeypatch.setattr(m, "LIB_PATH", str(tmp_path / "lib.so"))
    monkeypatch.setattr(m, "BINDING_PATH", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(m, "_compile", lambda out, extra=(): open(out, "w").close())
    (tmp_path / "bin").mkdir()

    def gxx(code):
        path = tmp_path / "bin" / "g++"
        path.write_text(GXX.format(code=code))
        path.chmod(0o755)
        monkeypatch.setenv("PATH", str(tmp_path / "bin") + os.pathsep + os.environ["PATH"])
    return tmp_path, gxx


def made(path):
    return sorted(os.path.basename(f).partition(".")[0] for f in glob.glob(str(path / "*.so*")))


def test_both_are_made(tree):
    path, gxx = tree
    gxx(0)
    assert m.build() == m.LIB_PATH and made(path) == ["_binding", "lib"]


def test_library_without_torch(tree, monkeypatch):
    path, gxx = tree
    gxx(0)
    monkeypatch.setitem(sys.modules, "torch", None)
    assert m.build() == m.LIB_PATH and made(path) == ["lib"]


def test_library_without_a_host_compiler(tree, monkeypatch):
    path, _ = tree
    monkeypatch.setenv("PATH", str(path / "bin"))
    assert m.build() == m.LIB_PATH and made(path) == ["lib"]


@pytest.mark.parametrize("what", ["python", "cuda"])
def test_library_without_headers(tree, monkeypatch, what):
    path, gxx = tree
    gxx(0)
    if what == "python":
        monkeypatch.setattr(sysconfig, "get_paths", lambda: {"include": str(path)})
    else:
        monkeypatch.setenv("CUDA_HOME", str(path))
    assert m.build() == m.LIB_PATH and made(path) == ["lib"]


def test_library_where_the_binding_fails(tree):
    path, gxx = tree
    gxx(3)
    with pytest.raises(subprocess.CalledProcessError):
        m.build()
    assert made(path) == ["lib"]


def test_binding_where_the_library_fails(tree, monkeypatch):
    path, gxx = tree

    def fails(out, extra=()):
        raise subprocess.CalledProcessError(1, "nvcc")
    monkeypatch.setattr(m, "_compile", fails)
    for code, left in ((3, []), (0, ["_binding"])):
        gxx(code)
        with pytest.raises(subprocess.CalledProcessError, match="nvcc"):
            m.build()
        assert made(path) == left


def test_no_binding_is_an_error_at_its_first_use(tree, monkeypatch):
    import torch

    from speculative_decoding_verify_03_gb300 import kv
    monkeypatch.setattr(kv, "_module", None)
    with pytest.raises(m.SpecError, match="build"):
        m.spec_tree_mask(torch.zeros((2, 3), dtype=torch.int32))


@pytest.mark.parametrize("change", ["torch", "python"])
def test_a_binding_made_for_another_torch_or_python_is_not_taken(tree, monkeypatch, change):
    """It is compiled against their interfaces, whatever the age of its own sources."""
    import torch

    from speculative_decoding_verify_03_gb300 import kv
    path, gxx = tree
    gxx(0)
    m.build()
    first = glob.glob(str(path / "_binding*"))
    assert len(first) == 1
    if change == "torch":
        monkeypatch.setattr(torch, "__version__", "9.9.9")
    else:
        monkeypatch.setattr(sysconfig, "get_config_var", lambda name: "cpython-999")
    monkeypatch.setattr(kv, "_module", None)
    with pytest.raises(m.SpecError, match="build"):
        m.spec_tree_mask(torch.zeros((2, 3), dtype=torch.int32))
    m.build()
    assert len(glob.glob(str(path / "_binding*"))) == 2
