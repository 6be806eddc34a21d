"""The build script away from its usual machine (CPU; no compiler runs)."""
import os
import sys

import pytest

from moe_grouped_gemm_block_amd import build


@pytest.fixture
def commands(monkeypatch, tmp_path):
    """The commands that build() would run; their outputs are empty files under tmp_path."""
    for name in ("LIB", "LIB_STAGES1", "BINDING"):
        monkeypatch.setattr(build, name, str(tmp_path / os.path.basename(getattr(build, name))))
    ran = []

    def run(cmd):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return ""

    monkeypatch.setattr(build, "_run", run)
    monkeypatch.setattr(build, "hipcc", lambda: "hipcc")
    return ran


def test_everything_is_built(commands, tmp_path):
    assert build.build(verbose=False) == build.LIB
    assert sorted(os.listdir(tmp_path)) == ["_dg_torch.so", "libdg.so", "libdg_stages1.so"]
    assert len(commands) == 2 * (len(build.SOURCES) + 1) + 1


def test_the_libraries_are_built_without_torch(commands, tmp_path, monkeypatch, capsys):
    """libdg.so is a C library: a machine with ROCm and no torch builds it, and is
    told that the torch binding is left out."""
    monkeypatch.setitem(sys.modules, "torch", None)             # importing it raises ImportError
    assert build.build(verbose=False) == build.LIB
    assert sorted(os.listdir(tmp_path)) == ["libdg.so", "libdg_stages1.so"]
    assert not any("binding.cpp" in a for c in commands for a in c)
    assert "torch" in capsys.readouterr().err


@pytest.mark.parametrize("abi", [True, False])
def test_the_binding_follows_torch_and_cxx(monkeypatch, abi):
    """The host compiler is the caller's, the C++ ABI torch's."""
    import torch
    monkeypatch.setenv("CXX", "some-c++")
    monkeypatch.setattr(torch, "compiled_with_cxx11_abi", lambda: abi)
    cmd = build.binding_command("out.so")
    assert cmd[0] == "some-c++" and f"-D_GLIBCXX_USE_CXX11_ABI={int(abi)}" in cmd
