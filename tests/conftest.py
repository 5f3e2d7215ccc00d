import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

# CPU tests that make valid calls on made-up addresses, to see them pass the
# checks and end in HKG_ERR_DEVICE: where there is a GPU they would be launched
VALID_CALLS_ON_MADE_UP_ADDRESSES = (
    "test_ops_abi.py::test_gemm_operands_may_alias",
    "test_abi.py::test_overlapping_outputs_rejected",
    "test_abi.py::test_row_pitches_validated_before_launch",
)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU; runs through the C ABI")
    config.addinivalue_line("markers", "slow: long-running CPU test")


# Tests that expect a launch to begin at XCD 0.  The hardware queue decides where it begins:
# at 0 until a process has used more streams than there are queues, at any XCD from then on
# (tests/test_gpu_xcd.py), so these run before every other test.
ON_THE_FIRST_QUEUE = ("test_workgroup_b_runs_on_xcd_b_mod_8", "test_time_record")


def first_queue_first(items):
    """`items` with the tests of ON_THE_FIRST_QUEUE in front, otherwise in their order."""
    return sorted(items, key=lambda i: i.name.split("[")[0] not in ON_THE_FIRST_QUEUE)


def pytest_collection_modifyitems(config, items):
    items[:] = first_queue_first(items)
    named = [i for i in items if i.nodeid.endswith(VALID_CALLS_ON_MADE_UP_ADDRESSES)]
    if not named:
        return
    try:
        import torch
    except ImportError:
        return
    if torch.cuda.is_available():
        for i in named:
            i.add_marker(pytest.mark.skip(reason="valid calls on made-up addresses: a GPU is present"))
