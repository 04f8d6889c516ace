"""What the build does with what it finds, without compiling anything."""
import sys

import pytest

from bigvgan_waveform_decoder_b200 import build as B


@pytest.fixture
def calls(monkeypatch):
    made = []
    monkeypatch.setattr(B, "build_library", lambda *a: made.append("library"))
    monkeypatch.setattr(B, "build_ops", lambda *a: made.append("operators"))
    return made


def test_library_and_operators(calls):
    assert B.build() == B.LIB and calls == ["library", "operators"]


def test_the_library_is_built_without_torch(calls, monkeypatch, capsys):
    """The decoder takes device pointers: only the operators' front end needs torch."""
    monkeypatch.setitem(sys.modules, "torch", None)  # an import fails as if it were not installed

    def needs_torch(*a):
        import torch  # noqa: F401

    monkeypatch.setattr(B, "build_ops", needs_torch)
    assert B.build() == B.LIB and calls == ["library"]
    assert "torch is not installed" in capsys.readouterr().err
