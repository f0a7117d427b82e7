"""CPU checks of what build() compiles again."""

import subprocess

import pytest

from split_kv_decode_bsr_gb300 import build as sta_build


def _commands(monkeypatch):
    """The commands of a build() in which the first ones fail."""
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        return subprocess.CompletedProcess(cmd, 1, "", "")

    with monkeypatch.context() as m:
        m.setattr(sta_build.subprocess, "run", run)
        try:
            sta_build.build()
        except RuntimeError:
            assert ran
    return ran


def test_the_binding_is_compiled_again_for_another_torch_or_python(monkeypatch):
    import sysconfig

    import torch

    sta_build.build()
    assert _commands(monkeypatch) == []
    soabi = sysconfig.get_config_var("SOABI")
    for change in (lambda m: m.setattr(torch, "__version__", "0.0.1"),
                   lambda m: m.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI),
                   lambda m: m.setattr(sysconfig, "get_config_var", lambda name: "other" if name == "SOABI" else soabi)):
        with monkeypatch.context() as m:
            change(m)
            ran = _commands(monkeypatch)
            assert len(ran) == 1 and any(a.endswith("bind.cpp") for a in ran[0])
    assert _commands(monkeypatch) == []
