"""The tests of hkg_linear.h's argument checks call the library on made-up addresses: none
of them may make a call that passes every check (tests/test_made_up_addresses.py says why,
and watches the other interfaces)."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)

PLUGIN = '''
import torch
import dense_gemm_fp8_amd as hkg
from dense_gemm_fp8_amd import linear16

torch.cuda.is_available = lambda: True
lib, reached = linear16._lib(), []


def watched(name):
    fn = getattr(lib, name)

    def call(*args):
        rc = fn(*args)
        if rc == hkg.HKG_ERR_DEVICE:
            reached.append(name)
        return rc
    return call


for name in linear16.LINEAR_EXPORTS:
    setattr(lib, name, watched(name))


def pytest_sessionfinish(session):
    print("\\nREACHED THE DEVICE: %r" % (reached,))
'''


@pytest.mark.skipif(torch.cuda.is_available(), reason="shown on a host without a GPU")
def test_no_call_on_a_made_up_address_reaches_the_device(tmp_path):
    (tmp_path / "watch_calls.py").write_text(PLUGIN)
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([str(tmp_path), ROOT]))
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "watch_calls", "-p", "no:cacheprovider",
                        os.path.join(HERE, "test_linear_abi.py")], cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    assert "REACHED THE DEVICE: []" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]
    assert " passed" in r.stdout
