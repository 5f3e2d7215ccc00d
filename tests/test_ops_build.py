"""Assembly checks of the operators' kernels (CPU): no load runs in a loop over
lane values, and the tiles' K loops hold nothing but their own instructions."""
import os
import re
import shutil

import pytest

from dense_gemm_fp8_amd import build

pytestmark = pytest.mark.skipif(not shutil.which(build.hipcc()), reason="hipcc not available")


def loops(asm):
    """{kernel: instructions of its loop with the most matrix instructions}."""
    out, fn, lines = {}, None, asm.splitlines()
    labels = {}
    for i, line in enumerate(lines):
        m = re.match(r"^(_Z\w+):", line)
        if m:
            fn, labels = m.group(1), {}
        m = re.match(r"^(\.LBB\w+):", line)
        if m:
            labels[m.group(1)] = i
        m = re.match(r"\s+s_cbranch\w*\s+(\.LBB\w+)", line)
        if m and m.group(1) in labels:
            body = [x.split()[0] for x in lines[labels[m.group(1)]:i] if x.startswith("\t") and x.strip()[0] not in ".;"]
            n = sum(x.startswith("v_mfma") for x in body)
            if n and n > sum(x.startswith("v_mfma") for x in out.get(fn, [])):
                out[fn] = body
    return out


@pytest.mark.parametrize("source,tiles", [("mxfp4_gemm.hip", "mx4_tile"), ("orth_kernels.hip", "orth_product"),
                                          ("mxfp4_kernels.hip", None)])
def test_kernels(tmp_path, source, tiles):
    out = os.path.join(tmp_path, "k.s")
    build.device_asm(out, source)
    asm = open(out).read()
    assert build.waterfall_loops(asm) == []
    if tiles is None:
        return
    found = {k: v for k, v in loops(asm).items() if tiles in k}
    assert len(found) >= 4
    for kernel, body in found.items():
        # an accumulator that moves between registers inside the loop costs more than
        # any load: the compiler does it where bookkeeping leaves its slot
        assert not any(x.startswith(("v_accvgpr", "scratch_")) for x in body), kernel
