"""What the build makes of the batch calls' tensor checks: a library of their
own, named by the torch and Python it reads tensors of, that a C program does
without."""
import os
import subprocess
import sys
import sysconfig

import pytest
import torch

from chunk_causal_attention_block_b200 import build as wfbuild
from chunk_causal_attention_block_b200 import wf


@pytest.fixture
def compiles(monkeypatch, tmp_path):
    """Commands that the build would run, which are not; libraries lie in a folder of their own."""
    ran = []
    monkeypatch.setattr(subprocess, "run", lambda cmd, **kw: ran.append(cmd))
    monkeypatch.setattr(wfbuild, "PKG", str(tmp_path))
    return ran


def test_the_name_carries_the_versions(monkeypatch, compiles):
    lib = wfbuild.torch_lib()
    assert torch.__version__.replace("+", "-") in lib and sysconfig.get_config_var("SOABI") in lib and lib.endswith(".so")
    wfbuild._build_torch_calls(False)
    assert [lib in cmd for cmd in compiles] == [True]
    with open(lib, "w"):
        pass
    wfbuild._build_torch_calls(False)
    assert len(compiles) == 1  # newer than its sources
    # after an upgrade the one at hand is not taken for built
    monkeypatch.setattr(torch, "__version__", "99.0")
    other = wfbuild.torch_lib()
    assert other != lib
    wfbuild._build_torch_calls(False)
    assert [other in cmd for cmd in compiles] == [False, True]


@pytest.mark.parametrize("newer", ["TORCH_SRC", "a header", "the flags"])
def test_it_is_built_again_for_what_it_is_made_of(monkeypatch, compiles, tmp_path, newer):
    lib = wfbuild.torch_lib()
    with open(lib, "w"):
        pass
    late = str(tmp_path / "newer")
    with open(late, "w"):
        pass
    os.utime(late, (os.path.getmtime(lib) + 10,) * 2)
    if newer == "TORCH_SRC":
        monkeypatch.setattr(wfbuild, "TORCH_SRC", late)
    elif newer == "a header":
        monkeypatch.setattr(wfbuild, "_headers", lambda: [late])
    else:
        monkeypatch.setattr(wfbuild, "__file__", late)
    wfbuild._build_torch_calls(False)
    assert [lib in cmd for cmd in compiles] == [True]


def test_a_library_for_another_torch_is_not_loaded(monkeypatch):
    monkeypatch.setattr(wf, "_torch_calls", None)
    monkeypatch.setattr(torch, "__version__", "99.0")
    with pytest.raises(RuntimeError, match="not built for this torch and Python .*99.0"):
        wf._batch_calls()
    monkeypatch.undo()
    assert wf._batch_calls() is not None


def test_no_torch_is_no_error(monkeypatch, compiles, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)  # importing it fails
    wfbuild._build_torch_calls(False)
    assert "no torch" in capsys.readouterr().err and not compiles


def test_no_gxx_is_no_error(monkeypatch, compiles, capsys):
    monkeypatch.setattr(wfbuild.shutil, "which", lambda name: None)
    wfbuild._build_torch_calls(False)
    assert "no g++" in capsys.readouterr().err and not compiles


def test_the_tensor_checks_can_be_left_out(monkeypatch):
    wfbuild.build()  # (all else is up to date then)
    asked = []
    monkeypatch.setattr(wfbuild, "_build_torch_calls", asked.append)
    assert wfbuild.build(torch_calls=False) == wfbuild.LIB and asked == []
    assert wfbuild.build() == wfbuild.LIB and asked == [False]
