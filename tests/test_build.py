"""The build step: the native argument checks belong to one torch and one Python."""
import pytest
import torch

from sparse_long_context_mse_b200 import api, build

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
