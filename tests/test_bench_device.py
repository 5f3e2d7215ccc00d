"""bench.metrics_reader reads the GPU that the benchmark runs on (CPU: amdsmi and
torch's device properties are stand-ins)."""
import sys
import types

import pytest

torch = pytest.importorskip("torch")

import bench  # noqa: E402


def smi(bdfs):
    m = types.ModuleType("amdsmi")
    m.amdsmi_init = lambda: None
    m.amdsmi_get_processor_handles = lambda: list(range(len(bdfs)))
    m.amdsmi_get_gpu_device_bdf = lambda h: bdfs[h]
    m.amdsmi_get_gpu_metrics_info = lambda h: {"mem_activity_acc": 10 * h, "gfx_activity_acc": 20 * h,
                                               "accumulation_counter": 30 * h, "vram_max_bandwidth": 8000}
    return m


@pytest.mark.parametrize("bus,read", [(0x05, (0, 0, 0, 8000)), (0xA7, (20, 40, 60, 8000)), (0x99, None)])
def test_reads_the_gpu_in_use_among_several(monkeypatch, bus, read):
    monkeypatch.setitem(sys.modules, "amdsmi", smi(["0000:05:00.0", "0000:15:00.0", "0000:A7:00.0"]))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "get_device_properties",
                        lambda d: types.SimpleNamespace(pci_domain_id=0, pci_bus_id=bus, pci_device_id=0))
    reader = bench.metrics_reader()
    assert (reader and reader()) == read
