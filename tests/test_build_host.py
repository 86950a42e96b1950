"""The build on machines other than the one it was first run on."""
import os
import sys

import pytest

from ternary_weight_bit_w2a8_b200 import build


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """A build whose binding lies in a folder of its own, and whose compiler calls are recorded instead of made."""
    build.build()
    calls = []

    def run(cmd, check=True):
        calls.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(build.subprocess, "run", run)
    return calls


def test_the_c_library_needs_no_torch(elsewhere, monkeypatch, capfd):
    monkeypatch.setitem(sys.modules, "torch", None)  # importing it fails
    assert build.build() == build.LIB
    assert not elsewhere and not os.path.exists(build.BINDING)
    assert "binding" in capfd.readouterr().err  # said, not passed over


def test_the_binding_is_built_where_torch_is(elsewhere):
    assert build.build() == build.LIB
    assert [c[0] for c in elsewhere] == ["g++"] and os.path.exists(build.BINDING)
    build.build()
    assert len(elsewhere) == 1  # it is up to date


def test_a_torch_without_cuda_is_none(elsewhere, monkeypatch, capfd):
    import torch
    monkeypatch.setattr(torch.version, "cuda", None)
    assert build.build() == build.LIB
    assert not elsewhere and "binding" in capfd.readouterr().err
