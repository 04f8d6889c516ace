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


def test_operators_are_built_again_for_another_torch(monkeypatch, tmp_path):
    """An _ops.so that is newer than its sources is up to date only for the torch and Python it was built for."""
    ops, runs = tmp_path / "_ops.so", []

    def run(cmd, check):
        runs.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass

    monkeypatch.setattr(B, "OPS", str(ops))
    monkeypatch.setattr(B, "OPS_STAMP", str(tmp_path / "made" / "_ops.stamp"), raising=False)
    monkeypatch.setattr(B.subprocess, "run", run)
    for _ in range(2):
        B.build_ops()
        assert len(runs) == 1 and ops.exists()
    B.build_ops(force=True)
    assert len(runs) == 2
    version = B.metadata.version
    monkeypatch.setattr(B.metadata, "version", lambda name: "9.9" if name == "torch" else version(name))
    for _ in range(2):
        B.build_ops()
        assert len(runs) == 3
    ops.unlink()
    B.build_ops()
    assert len(runs) == 4
