"""include/hkg_ops.h under AddressSanitizer and UndefinedBehaviorSanitizer (host code
only, on the CPU): tests/c/ops_extremes.c calls every entry point with extreme sizes
and pitches; a signed overflow in a check ends the run with a report."""
import os
import shutil
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.join(HERE, "c"))

import build_sanitized  # noqa: E402


@pytest.mark.skipif(not shutil.which("/opt/rocm/bin/hipcc"), reason="hipcc not available")
def test_ops_extremes_under_sanitizers(tmp_path, monkeypatch):
    monkeypatch.setattr(build_sanitized, "SRC", os.path.join(HERE, "c", "ops_extremes.c"))
    exe = build_sanitized.build(str(tmp_path / "ops_extremes"))
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600, env=env)
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
    assert "OPS EXTREMES OK" in r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr
