"""What the build leaves behind, with compilers that only write their output file (or fail)."""
import os

import pytest
import torch

import kda_linear_attention_bounded_gb300 as kda
from kda_linear_attention_bounded_gb300 import _hybrid
from kda_linear_attention_bounded_gb300 import build as kbuild

FAKE = """#!/bin/sh
echo "$0" >> "{log}"
while [ $# -gt 0 ]; do if [ "$1" = -o ]; then echo made > "$2"; fi; shift; done
"""


@pytest.fixture
def fake(tmp_path, monkeypatch):
    """Fake compilers and an empty build folder; the calls made so far."""
    log = tmp_path / "log"
    for name in ("nvcc", "g++"):
        (tmp_path / name).write_text(FAKE.format(log=log))
        (tmp_path / name).chmod(0o755)
    monkeypatch.setenv("NVCC", str(tmp_path / "nvcc"))
    monkeypatch.setenv("CXX", str(tmp_path / "g++"))
    monkeypatch.setattr(kbuild, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(kbuild, "LIB", str(tmp_path / "_build" / "libkda.so"))

    def calls():
        made = [os.path.basename(x) for x in log.read_text().split()] if log.exists() else []
        log.write_text("")
        return made.count("nvcc"), made.count("g++")

    return calls


def test_builds_once(fake):
    assert kbuild.build() == kbuild.LIB
    assert os.path.exists(kbuild.LIB) and os.path.exists(kbuild.torch_ext())
    assert fake() == (len(kbuild.sources()) + 1, 1)
    kbuild.build()
    assert fake() == (0, 0)
    kbuild.build(force=True)
    assert fake() == (len(kbuild.sources()) + 1, 1)


def test_another_torch_has_a_module_of_its_own(fake, monkeypatch):
    kbuild.build()
    fake()
    first = kbuild.torch_ext()
    monkeypatch.setattr(torch, "__version__", "0.0.1+test")
    assert kbuild.torch_ext() != first
    monkeypatch.setattr(_hybrid, "_ext", _hybrid._Unloaded())
    monkeypatch.setattr(_hybrid._b, "load", lambda: None)
    x = torch.zeros(1)
    with pytest.raises(RuntimeError, match="not built for this interpreter and torch"):
        kda.gdn_decode(x, x, x, x, x, x, x, x, x, out=x, workspace=x)
    kbuild.build()
    assert fake() == (0, 1)
    assert os.path.exists(first) and os.path.exists(kbuild.torch_ext())


@pytest.mark.parametrize("compiler", ["/bin/false", "/no/such/compiler"])
def test_library_without_the_binding(fake, monkeypatch, compiler):
    monkeypatch.setenv("CXX", compiler)
    assert kbuild.build(binding=False) == kbuild.LIB and os.path.exists(kbuild.LIB)
    assert not os.path.exists(kbuild.torch_ext())
    os.remove(kbuild.LIB)
    with pytest.raises(RuntimeError, match="kda_torch.cpp"):
        kbuild.build()
    assert os.path.exists(kbuild.LIB) and not os.path.exists(kbuild.torch_ext())   # the library is there all the same


def test_library_that_does_not_compile(fake, monkeypatch):
    monkeypatch.setenv("NVCC", "/bin/false")
    with pytest.raises(RuntimeError, match="kda_api.cu"):
        kbuild.build()
    assert not os.path.exists(kbuild.LIB)
