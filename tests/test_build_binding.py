"""When the paged cache's extension module is compiled, and when the library is
built without it (no compiler runs here)."""

import os
import types

import pytest

from gated_linear_sliding_chunkwise_b200 import build


@pytest.fixture
def fake(tmp_path, monkeypatch):
    """build_binding into an empty folder, with a compiler that only writes its output."""
    runs = []

    def run(cmd, **kw):
        runs.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("module")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_paged_call.so"))
    monkeypatch.setattr(build, "subprocess", types.SimpleNamespace(run=run))
    return runs


def test_the_module_is_compiled_once(fake):
    assert build.build_binding() == build.BINDING and len(fake) == 1
    assert build.build_binding() == build.BINDING and len(fake) == 1
    assert build.build_binding(force=True) == build.BINDING and len(fake) == 2


def test_another_torch_or_python_compiles_it_again(fake, monkeypatch):
    build.build_binding()
    monkeypatch.setattr(build, "_torch_version", lambda: "torch 0.0, python 3.0\n")
    build.build_binding()
    assert len(fake) == 2
    build.build_binding()
    assert len(fake) == 2


@pytest.mark.parametrize("what", ["torch", "g++", "cuda"])
def test_the_library_is_built_without_it(fake, monkeypatch, capsys, what):
    """Without torch, without g++ or with a torch for CPUs the library's build
    goes through, and no module for another torch stays behind."""
    build.build_binding()
    if what == "torch":
        monkeypatch.setattr(build, "_torch_version", lambda: None)
    elif what == "g++":
        which = build.shutil.which
        monkeypatch.setattr(build.shutil, "which", lambda name: None if name == "g++" else which(name))
    else:
        import torch
        monkeypatch.setattr(torch.version, "cuda", None)
    assert build.build_binding(force=True) is None and len(fake) == 1
    assert "left out" in capsys.readouterr().err
    assert not os.path.exists(build.BINDING)


def test_the_version_of_this_torch():
    import torch
    assert torch.__version__.split("+")[0] in build._torch_version()
