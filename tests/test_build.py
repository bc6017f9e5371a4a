"""What the build needs: nvcc for the C library, PyTorch only for its binding; and a binding of another PyTorch is
neither kept nor loaded.  The compilers are stand-ins here."""
import os
import subprocess
import sys
from pathlib import Path

import pytest

ROOT = Path(__file__).resolve().parent.parent


def compiler(calls):
    """A stand-in for subprocess.run: notes the command, and touches its -o."""

    def run(cmd, **kw):
        calls.append([str(c) for c in cmd])
        Path(calls[-1][calls[-1].index("-o") + 1]).touch()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    return run


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    from expert_ffn_gemv_b200 import build

    monkeypatch.setattr(build, "OUT_DIR", tmp_path)
    monkeypatch.setattr(build, "LIB", tmp_path / "libmoe_b200.so")
    monkeypatch.setattr(build, "EXT", tmp_path / "_block_ext.so")
    return build


def test_library_without_torch(tmp_path):
    """In a process that cannot import torch."""
    code = f"""
import sys
sys.path.insert(0, {str(ROOT)!r})
sys.path.insert(0, {str(ROOT / "tests")!r})
sys.modules["torch"] = None
from pathlib import Path
import expert_ffn_gemv_b200.build as b
from test_build import compiler
b.OUT_DIR = Path({str(tmp_path)!r})
b.LIB, b.EXT = b.OUT_DIR / "libmoe_b200.so", b.OUT_DIR / "_block_ext.so"
calls = []
b.subprocess.run = compiler(calls)
assert b.build() == b.LIB and b.LIB.exists() and not b.EXT.exists()
assert len(calls) == len(b.SOURCES) + 1 and not any("bind.cpp" in " ".join(c) for c in calls)
calls.clear()
assert b.build() == b.LIB and not calls
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, env={**os.environ, "PYTEST_DISABLE_PLUGIN_AUTOLOAD": "1"})
    assert r.returncode == 0, r.stderr


def test_binding_of_another_torch_is_built_again(elsewhere, monkeypatch):
    calls = []
    monkeypatch.setattr(elsewhere.subprocess, "run", compiler(calls))
    target = elsewhere.ext_target()
    for built_for, again in ((target, 0), (target + "1", 1), (None, 1)):
        text = b"" if built_for is None else b"moe-block-ext-for:" + built_for.encode() + b"\0"
        elsewhere.EXT.write_bytes(b"\x7fELF" + text + b"..")
        calls.clear()
        elsewhere.build_ext()
        assert len(calls) == again, built_for
        assert not again or any(target in c for c in calls[0])


def test_binding_of_another_torch_is_not_loaded(tmp_path):
    from expert_ffn_gemv_b200 import build

    build.build()
    from expert_ffn_gemv_b200 import block

    assert build.ext_built_for(build.EXT) == build.ext_target()
    other = tmp_path / "_block_ext.so"
    other.write_bytes(build.EXT.read_bytes().replace(build.ext_target().encode(), b"torch 0.0.0".ljust(len(build.ext_target()))))
    with pytest.raises(RuntimeError, match="built for torch 0.0.0"):
        block._load_ext(other)
    with pytest.raises(RuntimeError, match="missing"):
        block._load_ext(tmp_path / "none.so")
