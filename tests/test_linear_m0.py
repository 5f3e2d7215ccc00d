"""M0 in the linear layer's kernels (CPU): a load to LDS takes its LDS address from M0.  Beside
transposed operands M0 is set in one assembly statement and used in a later one, which does
not name it, so that nothing may write M0 in between; the listing shows whether anything does."""
import os
import re
import shutil

import pytest

from dense_gemm_fp8_amd import build


def m0_events(body):
    """(line, "set" | "load" | "other", text) of every instruction that writes M0 or uses it."""
    out = []
    for i, line in enumerate(x.split(";")[0].strip() for x in body.splitlines()):
        if re.match(r"buffer_load\S* .*\blds$", line):
            out.append((i, "load", line))
        elif re.match(r"s_add_u32 m0,", line):
            out.append((i, "set", line))
        elif re.search(r"\bm0\b", line):
            out.append((i, "other", line))
    return out


def out_of_order(body):
    """What is wrong: each load has to follow a set of its own, an instruction at least between
    them (the wait state that the hardware asks for), with no label that a branch could enter by."""
    lines, wrong, last = body.splitlines(), [], None
    for i, what, text in m0_events(body):
        if what == "load":
            if last is None or i - last < 2:
                wrong.append((i, text))
            elif any(re.match(r"\s*[.\w$]+:", x) for x in lines[last:i]):
                wrong.append((i, "label before " + text))
            last = None
        elif what == "set" and last is None:
            last = i
        else:
            wrong.append((i, text))
    return wrong


def test_the_check_itself():
    good = "\ts_add_u32 m0, s1, 4096\n\tv_mfma_f32 a, b\n\tbuffer_load_dwordx4 v1, s[0:3], s4 offen lds\n"
    assert out_of_order(good * 3) == []
    one, two, three = good.splitlines(True)
    assert out_of_order(one + three)                                   # no instruction between
    assert out_of_order(two + three)                                   # not set
    assert out_of_order(one + two + three + two + three)               # set once for two loads
    assert out_of_order(one + two + "\ts_mov_b32 m0, s7\n" + three)    # written by something else
    assert out_of_order(one + two + ".LBB0_1:\n" + three)              # entered between
    assert out_of_order(one + two + one + two + three)                 # two sets


@pytest.mark.skipif(not shutil.which(build.hipcc()), reason="hipcc not available")
def test_m0_between_set_and_load(tmp_path):
    path = os.path.join(tmp_path, "k.s")
    build.device_asm(path, "linear_gemm.hip")
    bodies = re.findall(r"^(_Z\w*linear_\w+_kernel\w*):(.*?)^\.Lfunc_end", open(path).read(), re.S | re.M)
    seen = 0
    for name, body in bodies:
        if "ds_read_b64_tr_b16" not in body:
            continue
        seen += 1
        assert len([1 for e in m0_events(body) if e[1] == "load"]) >= 24, name
        assert out_of_order(body) == [], name
    assert seen >= 20
