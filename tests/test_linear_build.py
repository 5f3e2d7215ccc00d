"""Assembly checks of the linear layer's kernels (CPU), as tests/test_ops_build.py and
tests/test_ops_lane_order.py make them of the others: no accumulator moves inside the K
loops, no load runs in a loop over lane values, no wait for all loads before a transposed
read, and where lanes read what other lanes staged the compiler has been told so."""
import os
import re
import shutil

import pytest

from dense_gemm_fp8_amd import build
from test_ops_build import loops

pytestmark = pytest.mark.skipif(not shutil.which(build.hipcc()), reason="hipcc not available")


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    out = {}
    for source in ("linear_gemm.hip", "linear_kernels.hip"):
        path = os.path.join(tmp_path_factory.mktemp("asm"), "k.s")
        build.device_asm(path, source)
        out[source] = open(path).read()
    return out


@pytest.mark.parametrize("source", ["linear_gemm.hip", "linear_kernels.hip"])
def test_no_load_in_a_loop_over_lane_values(asm, source):
    assert build.waterfall_loops(asm[source]) == []


def test_no_packed_fp32(asm):
    for text in asm.values():
        assert not re.search(r"\bv_pk_(add|mul|fma)_f32\b", text)


def test_k_loops(asm):
    found = {k: v for k, v in loops(asm["linear_gemm.hip"]).items() if "linear_tile" in k or "linear_part" in k}
    assert len(found) >= 20
    for kernel, body in found.items():
        assert not any(x.startswith(("v_accvgpr", "scratch_")) for x in body), kernel


def test_transposed_reads_do_not_wait_for_loads(asm):
    bodies = re.findall(r"^(_Z\w*linear_\w+_kernel\w*):(.*?)^\.Lfunc_end", asm["linear_gemm.hip"], re.S | re.M)
    seen = 0
    for name, body in bodies:
        if "ds_read_b64_tr_b16" not in body:
            continue
        seen += 1
        lines = [x.strip() for x in body.splitlines()]
        first, last = (f(i for i, x in enumerate(lines) if x.startswith("v_mfma")) for f in (min, max))
        # in the K loop the only waits for loads are the loop's own, of what is in flight
        waits = [x for x in lines[first:last] if "vmcnt(0)" in x]
        assert not waits, name
    assert seen >= 8


def test_staged_rows_are_read_behind_a_wave_barrier(asm):
    bodies = re.findall(r"^(_Z\w*linear_tile\w*):(.*?)^\.Lfunc_end", asm["linear_gemm.hip"], re.S | re.M)
    assert len(bodies) >= 10
    for name, body in bodies:
        assert body[body.rindex("v_mfma"):].count("; wave barrier") >= 4, name
