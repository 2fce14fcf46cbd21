"""The build where torch is missing or another one than before (host only)."""
import os
import sys

import pytest

from moe_expert_layer_sorted_gb300 import _build


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """The library is up to date; the binding would go to an empty folder."""
    _build.build()
    monkeypatch.setattr(_build, "BINDING", str(tmp_path / "_kv_binding.so"))
    return tmp_path


def test_the_library_builds_without_torch(elsewhere, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)  # not importable
    assert _build.build() == _build.LIB
    assert not os.listdir(elsewhere)


def test_the_binding_is_built_again_for_another_torch(elsewhere, monkeypatch):
    built = []

    def command(out, lib=None):
        built.append(out)
        return ["touch", out]

    monkeypatch.setattr(_build, "_binding_cmd", command)
    _build.build()
    _build.build()
    assert len(built) == 1
    monkeypatch.setattr(_build, "_binding_for", lambda: "torch 0.0")
    _build.build()
    _build.build()
    assert len(built) == 2
