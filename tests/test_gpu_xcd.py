"""Where the workgroups of a launch run, on any stream: round the 8 XCDs in turn, from one
that the hardware queue decides.  The grid remap needs no more than that."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("no GPU", allow_module_level=True)

import dense_gemm_fp8_amd as hkg  # noqa: E402

G = 4096


def check(record):
    xcd = record.cpu().numpy()[:, 0] & 0xF
    assert xcd.max() < 8
    np.testing.assert_array_equal((xcd - xcd[0]) % 8, np.arange(G) % 8)


@pytest.mark.parametrize("full_lds", [True, False])
def test_workgroups_go_round_the_xcds_on_every_stream(full_lds):
    """More streams than a process has hardware queues, and the default one afterwards."""
    for stream in [torch.cuda.Stream() for _ in range(9)] + [None]:
        with torch.cuda.stream(stream):
            record = hkg.probe_xcd(G, full_lds, 0)
        torch.cuda.synchronize()
        check(record)


def test_and_in_a_replayed_graph():
    hkg.probe_xcd(G, True, 0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        record = hkg.probe_xcd(G, True, 0)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        check(record)
