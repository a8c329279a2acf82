"""When the tensor binding is built again."""
import os
import subprocess

import pytest

from precision_activation_quantization_b200 import build


@pytest.fixture
def built(tmp_path, monkeypatch):
    """A binding that a stand-in for the compiler makes; yields how often it ran."""
    runs = []

    def compiler(cmd, **_):
        runs.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("binding")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_pqg_torch.so"))
    monkeypatch.setattr(build, "BINDING_ABI", str(tmp_path / "_pqg_torch.abi"), raising=False)
    monkeypatch.setattr(build.subprocess, "run", compiler)
    build.build_binding()
    assert len(runs) == 1
    return runs


def test_a_binding_of_this_torch_is_kept(built):
    build.build_binding()
    assert len(built) == 1
    build.build_binding(force=True)
    assert len(built) == 2


def test_a_binding_of_another_torch_is_built_again(built, monkeypatch):
    import torch
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    build.build_binding()
    assert len(built) == 2
    build.build_binding()
    assert len(built) == 2


def test_a_binding_of_unknown_origin_is_built_again(built):
    os.remove(build.BINDING_ABI)
    build.build_binding()
    assert len(built) == 2


def test_newer_sources_build_it_again(built):
    before = os.path.getmtime(build.BINDING_SRC) - 10
    os.utime(build.BINDING, (before, before))
    build.build_binding()
    assert len(built) == 2
