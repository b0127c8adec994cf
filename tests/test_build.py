"""The build step: the native argument checks belong to one torch and one Python, and the
C library needs neither."""
import os
import subprocess
import sys

import pytest
import torch

from sparse_long_context_mse_b200 import api, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_checks_built_for_another_torch_are_not_used(monkeypatch):
    build.build()
    assert not build._binding_stale()
    api._native()
    monkeypatch.setattr(torch, "__version__", "99.0.0+cu999")
    assert build._binding_stale()
    monkeypatch.setattr(api, "_binding", None)
    with pytest.raises(RuntimeError, match="missing"):
        api._native()


def test_checks_built_for_another_python_are_not_used(monkeypatch):
    build.build()
    real = build.sysconfig.get_config_var
    monkeypatch.setattr(build.sysconfig, "get_config_var",
                        lambda k: ".cpython-399-x86_64-linux-gnu.so" if k == "EXT_SUFFIX" else real(k))
    assert build._binding_stale()


def test_the_library_builds_without_torch():
    build.build()
    code = ("import sys; sys.modules['torch'] = None\n"
            "from sparse_long_context_mse_b200 import build as b\n"
            "if hasattr(b, 'BINDING'): b.BINDING += '.absent'\n"
            "assert b.build() == b.LIB and b.up_to_date()\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert "not built" in r.stderr
