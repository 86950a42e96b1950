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


@pytest.mark.parametrize("name,value", [("torch", "0.1"), ("python", "cpython-27")])
def test_another_torch_or_python_needs_another_binding(elsewhere, monkeypatch, name, value):
    import torch
    build.build()
    assert len(elsewhere) == 1
    if name == "torch":
        monkeypatch.setattr(torch, "__version__", value)
    else:
        monkeypatch.setattr(sys.implementation, "cache_tag", value)
    build.build()
    assert len(elsewhere) == 2
    build.build()
    assert len(elsewhere) == 2


def test_a_binding_of_another_torch_is_not_loaded():
    """In a process of its own: the module refuses to be initialised, and says why."""
    import subprocess
    from conftest import ROOT
    build.build()
    code = ("import torch\ntorch.__version__ = '0.1'\n"
            "import ternary_weight_bit_w2a8_b200 as bn\n"
            "try:\n    bn.bitnet_fp4_quant(torch.zeros(1, 4), 0)\n"
            "except ImportError as e:\n    print('refused:', e)\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.startswith("refused:") and "0.1" in r.stdout and "build" in r.stdout
