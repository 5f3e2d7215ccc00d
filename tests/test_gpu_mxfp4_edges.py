"""GPU tests of the MXFP4 operators at sizes where there is nothing to sum."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("no GPU", allow_module_level=True)

import dense_gemm_fp8_amd as hkg  # noqa: E402


def codes(rows, k):
    return torch.zeros((rows, k // 2), dtype=torch.uint8, device="cuda")


NONE = torch.zeros(0, dtype=torch.uint8, device="cuda")


# few rows, 128-tiles, 256-tiles, 256-tiles in two launches
@pytest.mark.parametrize("M,N", [(3, 5), (64, 2000), (2048, 1024), (1500, 1300), (4200, 4000), (4300, 14300), (100000, 16)])
def test_product_over_no_k_is_zero(M, N):
    C = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    F = torch.full((M, N), float("nan"), dtype=torch.float32, device="cuda")
    hkg.gemm_mxfp4(codes(M, 0), codes(N, 0), NONE, NONE, C, F)
    assert not C.any() and not F.any()
    y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    hkg.linear_mxfp4(torch.zeros((M, 0), dtype=torch.bfloat16, device="cuda"), codes(N, 0), NONE, y=y)
    assert not y.any()


@pytest.mark.parametrize("M,N,K", [(5, 0, 7), (2048, 0, 1024), (4200, 0, 4352), (0, 5, 7), (0, 2048, 1024), (0, 4300, 14300)])
def test_gradients_over_nothing_are_zero(M, N, K):
    dx = torch.full((M, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    dw = torch.full((N, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide = lambda n: -(-n // 32) * 32  # noqa: E731
    one = lambda n: torch.full((-(-K // 128) * -(-n // 128) * 512,), 127, dtype=torch.uint8, device="cuda")  # noqa: E731
    hkg.linear_mxfp4_backward(torch.zeros((M, N), dtype=torch.bfloat16, device="cuda"), codes(K, wide(N)), one(N),
                              codes(K, wide(M)), one(M), dx, dw)
    assert not dx.any() and not dw.any()


def test_linear_with_more_columns_than_one_launch_takes():
    """N = 2^28 + 200: 2^23 workgroups of 512 threads and more for one row of x.  W repeats
    2^20 rows of codes; its scales are 2^(g mod 3) for the 128 rows of group g."""
    N, K, period = (1 << 28) + 200, 32, 1 << 20
    g = torch.Generator("cuda").manual_seed(3)
    some = torch.randint(0, 256, (period, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    W = torch.empty((N, K // 2), dtype=torch.uint8, device="cuda")
    for r in range(0, N, period):
        W[r:r + period].copy_(some[:N - r])
    groups = -(-N // 128)
    exponent = torch.arange(groups, device="cuda") % 3
    packed = (127 + exponent).to(torch.uint8)[:, None].expand(groups, 512).contiguous().view(-1)
    x = torch.tensor([[0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0] * 4], device="cuda").to(torch.bfloat16)   # its own MXFP4 form
    y = torch.full((1, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    hkg.linear_mxfp4(x, W, packed, y=y)
    one = torch.full((period // 128 * 512,), 127, dtype=torch.uint8, device="cuda")
    values = hkg.mxfp4_dequantize(some, one, hkg.HKG_MX_OPERAND_B, dtype=torch.float32)
    want = values.double() @ x[0].double()             # multiples of 1/4 below 2^11: exact in fp32
    for r in range(0, N, period):
        n = min(period, N - r)
        e = exponent[r // 128:-(-(r + n) // 128)].repeat_interleave(128)[:n]
        assert torch.equal(y[0, r:r + n], (want[:n] * torch.exp2(e.double())).float().to(torch.bfloat16))
