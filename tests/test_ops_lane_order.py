"""Assembly check (CPU): where the tile kernels hand results from lane to lane through
LDS, the compiler has been told so.  After the K loop a wave stages rows of results and
its other lanes read them, with no workgroup barrier between: each such place holds a
wave barrier, which is no instruction but stops the compiler from moving the reads."""
import os
import re
import shutil

import pytest

from dense_gemm_fp8_amd import build

pytestmark = pytest.mark.skipif(not shutil.which(build.hipcc()), reason="hipcc not available")


@pytest.mark.parametrize("source,kernel", [("mxfp4_gemm.hip", "mx4_tile"), ("orth_kernels.hip", "orth_product")])
def test_staged_rows_are_read_behind_a_wave_barrier(tmp_path, source, kernel):
    out = os.path.join(tmp_path, "k.s")
    build.device_asm(out, source)
    bodies = re.findall(r"^(_Z\w*%s\w*):(.*?)s_endpgm" % kernel, open(out).read(), re.S | re.M)
    assert len(bodies) >= 4
    for name, body in bodies:
        epilogue = body[body.rindex("v_mfma"):]
        edge = int(re.search(r"ILi(256|192|128)E", name).group(1))
        # one for each 16 rows of the wave's quarter, at least
        assert epilogue.count("; wave barrier") >= edge // 32, name
