"""What the build makes of what: the library from nvcc alone, the Python binding
beside it for one Python and one torch.  The compilers are replaced."""
import importlib.util
import os
import sys

import pytest
import torch

from sparse_attention_prefill_cp_gb300 import _lib, build as B


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A tree of its own to build in, and compilers that write what they are asked for; those of ``refused`` fail."""
    pkg, csrc = tmp_path / "pkg", tmp_path / "pkg" / "csrc"
    csrc.mkdir(parents=True)
    for name in ("a.cu", "b.cu", "binding.cpp"):
        (csrc / name).write_text("")
    monkeypatch.setattr(B, "PKG_DIR", str(pkg))
    monkeypatch.setattr(B, "CSRC", str(csrc))
    monkeypatch.setattr(B, "BUILD_DIR", str(tmp_path / "_build"))
    monkeypatch.setattr(B, "LIB_PATH", str(pkg / "libdsa_cp.so"))
    monkeypatch.setattr(B, "nvcc", lambda: "/cuda/bin/nvcc")
    made, refused = [], set()

    class Compiler:
        def __init__(self, cmd, **kw):
            self.target = cmd[cmd.index("-o") + 1]
            self.returncode = int(any(r in " ".join(cmd) for r in refused))
            if not self.returncode:
                made.append(os.path.basename(self.target))
                open(self.target, "w").close()
            self.stdout = b"no such header"

        def communicate(self):
            return self.stdout, None

    monkeypatch.setattr(B.subprocess, "Popen", Compiler)
    monkeypatch.setattr(B.subprocess, "run", Compiler)
    return pkg, made, refused


def test_the_library_needs_no_binding(tree):
    pkg, made, refused = tree
    refused.add("binding.cpp")
    with pytest.raises(RuntimeError, match="no such header"):
        B.build()
    assert (pkg / "libdsa_cp.so").exists() and not list(pkg.glob("_binding*"))
    refused.clear()
    del made[:]
    B.build()
    assert len(list(pkg.glob("_binding*.so"))) == 1
    assert not any(name.startswith(("libdsa_cp", "a.", "b.")) for name in made)     # nothing of the library again


def test_a_tree_without_torch_builds_the_library(tree, monkeypatch):
    pkg, made, _ = tree
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert B.build() == str(pkg / "libdsa_cp.so")
    assert (pkg / "libdsa_cp.so").exists() and not list(pkg.glob("_binding*"))


def test_a_torch_that_cannot_be_imported_spoils_the_binding_alone(tree, monkeypatch):
    pkg, _, _ = tree

    def tag():
        raise ImportError("no such library")

    monkeypatch.setattr(B, "binding_tag", tag)
    with pytest.raises(ImportError, match="no such library"):
        B.build()
    assert (pkg / "libdsa_cp.so").exists()


def test_the_librarys_faults_are_raised(tree):
    pkg, _, refused = tree
    refused.add("b.cu")
    with pytest.raises(RuntimeError, match="b.cu"):
        B.build()
    assert not (pkg / "libdsa_cp.so").exists() and not list(pkg.glob("_binding*.so"))


def test_another_torch_gets_a_binding_of_its_own(tree, monkeypatch):
    pkg, made, _ = tree
    B.build()
    first = B.binding_path()
    assert sys.implementation.cache_tag in first and torch.__version__ in first and os.path.exists(first)
    monkeypatch.setattr(torch, "__version__", "99.1")
    assert B.binding_path() != first and not os.path.exists(B.binding_path())
    # asked for by a process that has loaded the library: built, and the library's file stays the one it loaded
    before = os.stat(pkg / "libdsa_cp.so")
    os.utime(pkg / "csrc" / "a.cu")
    monkeypatch.setattr(_lib, "_BINDING", None)
    monkeypatch.setattr(_lib, "load", lambda: None)
    with pytest.raises(ImportError):                 # the compilers of this test write empty files
        _lib.binding()
    assert os.path.exists(B.binding_path())
    after = os.stat(pkg / "libdsa_cp.so")
    assert (before.st_ino, before.st_mtime_ns) == (after.st_ino, after.st_mtime_ns)


def test_nothing_is_built_twice(tree):
    _, made, _ = tree
    B.build()
    assert len(made) == 5
    B.build()
    assert len(made) == 5
    B.build(force=True)
    assert len(made) == 10
