"""The compiled half of the binding fits one torch and one Python: it is built
again when either changes, and refused under another."""
import sysconfig

import pytest
import torch

from channel_pruned_decode_b200 import binding as B
from channel_pruned_decode_b200 import build


@pytest.fixture(autouse=True)
def built():
    build.build()


def test_built_again_for_another_torch_or_python(monkeypatch):
    assert not build.calls_stale()
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "1.0.0")
        assert build.calls_stale()
    with monkeypatch.context() as m:
        m.setattr(sysconfig, "get_config_var", lambda name: "cpython-39-other")
        assert build.calls_stale()
    with monkeypatch.context() as m:
        m.setattr(build, "CALLS_TAG", build.CALLS_TAG + ".missing")
        assert build.calls_stale()
    assert not build.calls_stale()


def test_refused_under_another_torch(monkeypatch):
    B._native()
    monkeypatch.setattr(B, "_calls", None)
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "1.0.0")
        with pytest.raises(RuntimeError, match="built for"):
            B._native()
    assert B._native().built_for == build.calls_tag()
