"""hkg_linear's workspace on the CPU: a size whose K is split over workgroups needs one, and
each refusal of it has its status, before any launch."""
import pytest

import dense_gemm_fp8_amd as hkg
from dense_gemm_fp8_amd import linear16 as lin

M, N, K = 100, 4096, 14336
G = 1 << 36                                  # distinct fake buffers, 64 GiB apart, never read
X, W, Y, WS, Z, R, BIAS, RNG = (i * G for i in range(1, 9))


def need(m=M, n=N, k=K):
    return lin._lib().hkg_linear_workspace_bytes(m, n, k)


def linear(ws=WS, n=None, e=None, m=M, y=Y):
    return lin._lib().hkg_linear(m, N, K, 0, X, 0, W, 0, e, y, 0, 0, ws, need() if n is None else n, None)


def epilogue(z=None, r=None, bias=None, rng=None):
    return lin.hkg_epilogue(bias, 0, 0, r, 0, z, 0, lin.hkg_dropout_opts(0.5 if rng else 0.0, 0, 0, rng))


def test_the_size_is_that_of_whole_tiles_of_sums():
    n = need()
    assert n > 0 and n % (4 * 128 * 128 * 32) == 0          # 32 tiles of 128, a number of parts
    assert need(1) == 0 and need(16) == 0 and need(0) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(ws=None), hkg.HKG_ERR_NULL), (dict(ws=WS + 8), hkg.HKG_ERR_ALIGN), (dict(n=0), hkg.HKG_ERR_WORKSPACE),
    (dict(n=-1), hkg.HKG_ERR_WORKSPACE), (dict(ws=Y), hkg.HKG_ERR_OVERLAP), (dict(ws=X), hkg.HKG_ERR_OVERLAP),
    (dict(ws=W + 16), hkg.HKG_ERR_OVERLAP), (dict(ws=Y + 2 * M * N - 16), hkg.HKG_ERR_OVERLAP),
    (dict(e=epilogue(z=WS + 64)), hkg.HKG_ERR_OVERLAP), (dict(e=epilogue(r=WS + 64)), hkg.HKG_ERR_OVERLAP),
    (dict(e=epilogue(bias=WS + 64)), hkg.HKG_ERR_OVERLAP), (dict(e=epilogue(rng=WS + 64)), hkg.HKG_ERR_OVERLAP),
])
def test_refusals(kw, status):
    assert linear(**kw) == status


def test_one_byte_short():
    assert linear(n=need() - 1) == hkg.HKG_ERR_WORKSPACE
    assert linear(ws=Y - need() + 16) == hkg.HKG_ERR_OVERLAP


def test_gradients_one_byte_short():
    n = lin._lib().hkg_linear_backward_workspace_bytes(64, 64, 64)
    args = (64, 64, 64, 0, X, 0, 0, W, 0, Z, 0, None, 0, 0, None, Y, 0, R, 0, None, WS)
    assert lin._lib().hkg_linear_backward(*args, n - 1, None) == hkg.HKG_ERR_WORKSPACE
