"""The tests of argument checks call the library on made-up addresses.  Where a
GPU is present none of them may make a call that passes every check: it would
be launched.  Here (no GPU) such a call ends in HKG_ERR_DEVICE, so the tests are
run with torch reporting a GPU and every call's status is recorded."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)

PLUGIN = '''
import pytest, torch
import dense_gemm_fp8_amd as hkg
from dense_gemm_fp8_amd import ops

torch.cuda.is_available = lambda: True
lib, now, reached = ops._lib(), [""], []


def watched(name):
    fn = getattr(lib, name)

    def call(*args):
        rc = fn(*args)
        if rc == hkg.HKG_ERR_DEVICE:
            reached.append(now[0] + ": " + name)
        return rc
    return call


for name in ops.OPS_EXPORTS + tuple(hkg.EXPORTS):
    setattr(lib, name, watched(name))


def pytest_runtest_setup(item):
    now[0] = item.nodeid


def pytest_sessionfinish(session):
    print("\\nREACHED THE DEVICE: %r" % (reached,))
'''


@pytest.mark.skipif(torch.cuda.is_available(), reason="shown on a host without a GPU")
def test_no_call_on_a_made_up_address_reaches_the_device(tmp_path):
    (tmp_path / "watch_calls.py").write_text(PLUGIN)
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([str(tmp_path), ROOT]))
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "watch_calls", "-p", "no:cacheprovider",
                        os.path.join(HERE, "test_abi.py"), os.path.join(HERE, "test_ops_abi.py")],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    assert "REACHED THE DEVICE: []" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]
    assert " passed" in r.stdout
