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
def compiles(monkeypatch):
    """Commands that the build would run, which are not."""
    ran = []
    monkeypatch.setattr(subprocess, "run", lambda cmd, **kw: ran.append(cmd))
    return ran


def test_the_name_carries_the_versions(monkeypatch, compiles):
    lib = wfbuild.torch_lib()
    assert torch.__version__.replace("+", "-") in lib and sysconfig.get_config_var("SOABI") in lib and lib.endswith(".so")
    assert os.path.exists(lib)
    wfbuild.build()
    assert not any(lib in cmd for cmd in compiles)  # up to date
    # after an upgrade the one at hand is not taken for built
    monkeypatch.setattr(torch, "__version__", "99.0")
    other = wfbuild.torch_lib()
    assert other != lib
    wfbuild.build()
    assert [other in cmd for cmd in compiles] == [True]


def test_a_library_for_another_torch_is_not_loaded(monkeypatch):
    monkeypatch.setattr(wf, "_torch_calls", None)
    monkeypatch.setattr(torch, "__version__", "99.0")
    with pytest.raises(RuntimeError, match="not built for this torch and Python .*99.0"):
        wf._batch_calls()
    monkeypatch.undo()
    assert wf._batch_calls() is not None


def test_libwf_is_built_without_torch(monkeypatch, compiles, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)  # importing it fails
    assert wfbuild.build() == wfbuild.LIB
    assert "no torch" in capsys.readouterr().err and not compiles


def test_libwf_is_built_without_gxx(monkeypatch, compiles, capsys):
    monkeypatch.setattr(torch, "__version__", "99.0")  # (to be built, that is)
    monkeypatch.setattr(wfbuild.shutil, "which", lambda name: None)
    assert wfbuild.build() == wfbuild.LIB
    assert "no g++" in capsys.readouterr().err and not compiles


def test_the_tensor_checks_can_be_left_out(monkeypatch, compiles):
    monkeypatch.setattr(torch, "__version__", "99.0")
    assert wfbuild.build(torch_calls=False) == wfbuild.LIB
    assert not compiles
