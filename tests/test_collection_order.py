"""Which tests run first (CPU): those that expect a launch to begin at XCD 0 hold on a
process's first hardware queue only."""
import os
import re

import conftest

HERE = os.path.dirname(os.path.abspath(__file__))


class Item:
    def __init__(self, name):
        self.name = name


def test_tests_of_the_first_queue_run_first():
    names = ["test_runs", "test_workgroup_b_runs_on_xcd_b_mod_8[True-0]", "test_runs[b]", "test_time_record[bf16-1]", "test_time_recorder"]
    got = [i.name for i in conftest.first_queue_first([Item(n) for n in names])]
    assert got == [names[1], names[3], names[0], names[2], names[4]]


def test_they_exist():
    text = open(os.path.join(HERE, "test_gpu_gemm.py")).read()
    for name in conftest.ON_THE_FIRST_QUEUE:
        assert re.search(r"^def %s\(" % name, text, re.M), name


def test_the_hook_orders_a_collection():
    class Config:
        pass
    items = [Item("test_linear"), Item("test_time_record[x]")]
    for i in items:
        i.nodeid = "tests/test_gpu_gemm.py::" + i.name
    conftest.pytest_collection_modifyitems(Config(), items)
    assert [i.name for i in items] == ["test_time_record[x]", "test_linear"]
