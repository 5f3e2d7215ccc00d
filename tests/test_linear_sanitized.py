"""include/hkg_linear.h under AddressSanitizer and UndefinedBehaviorSanitizer (host code
only, on the CPU): tests/c/linear_extremes.c calls every entry point with extreme sizes
and pitches; a signed overflow in a check, or a division by zero, ends the run."""
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.join(HERE, "c"))

import build_sanitized  # noqa: E402


@pytest.mark.skipif(not shutil.which("/opt/rocm/bin/hipcc"), reason="hipcc not available")
def test_linear_extremes_under_sanitizers(tmp_path, monkeypatch):
    monkeypatch.setattr(build_sanitized, "SRC", os.path.join(HERE, "c", "linear_extremes.c"))
    exe = str(tmp_path / "linear_extremes")
    *compiles, link = build_sanitized.commands(exe, str(tmp_path))

    def run(cmd):
        subprocess.run(cmd, check=True, stdout=subprocess.DEVNULL, stderr=subprocess.PIPE)

    with ThreadPoolExecutor(4) as pool:
        list(pool.map(run, compiles))
    run(link)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600, env=env)
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
    assert "LINEAR EXTREMES OK" in r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr
