"""The build's own rules, with the compilers replaced by one that only touches its output."""

import sys
from pathlib import Path

import pytest

from bit_block_quantized_q4_amd import build as b


@pytest.fixture
def fake(monkeypatch, tmp_path):
    """The build in tmp_path; the commands it ran."""
    ran = []

    def run(cmd, verbose):
        ran.append(cmd)
        Path(cmd[cmd.index("-o") + 1]).touch()

    monkeypatch.setattr(b, "_run", run)
    monkeypatch.setattr(b, "BUILD_DIR", tmp_path / "_build")
    for name in ("LIB_PATH", "HOST_LIB_PATH", "FLOOR_LIB_PATH", "TRACE_LIB_PATH", "TORCH_LIB_PATH"):
        monkeypatch.setattr(b, name, tmp_path / getattr(b, name).name)
    return ran


def torch_commands(ran):
    return [c for c in ran if str(b.TORCH_SRC) in c]


def test_the_library_builds_without_torch(fake, monkeypatch):
    b.TORCH_LIB_PATH.touch()  # of an earlier build
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch: ImportError
    assert b.build() == b.LIB_PATH
    for p in (b.LIB_PATH, b.HOST_LIB_PATH, b.FLOOR_LIB_PATH, b.TRACE_LIB_PATH):
        assert p.exists(), p
    assert not torch_commands(fake) and not b.TORCH_LIB_PATH.exists()


def test_the_library_builds_without_headers(fake, monkeypatch, tmp_path):
    import sysconfig
    monkeypatch.setattr(sysconfig, "get_paths", lambda: {"include": str(tmp_path / "none")})
    assert b.build() == b.LIB_PATH and b.LIB_PATH.exists()
    assert not torch_commands(fake) and not b.TORCH_LIB_PATH.exists()


def test_the_binding_is_built_behind_the_library(fake):
    pytest.importorskip("torch")
    b.build()
    assert b.TORCH_LIB_PATH.exists() and fake[-1] in torch_commands(fake)
    assert any(str(b.LIB_PATH.with_suffix(".so.tmp")) in c for c in fake[:-1])
