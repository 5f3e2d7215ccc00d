"""Host side of include/hkg_ops.h on the CPU: the library exports what the
header declares, and every refusal happens before any launch."""
import os
import re

import pytest

import dense_gemm_fp8_amd as hkg
from dense_gemm_fp8_amd import ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
G = 1 << 30                                  # distinct fake buffers, 1 GiB apart, never read
P = [i * G for i in range(1, 12)]
BIG = 1 << 40


def lib():
    return ops._lib()


def test_library_exports_every_declared_symbol():
    text = open(os.path.join(ROOT, "include", "hkg_ops.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(hkg_[a-z0-9_]+)\s*\(", text)))
    assert sorted(ops.OPS_EXPORTS) == names
    for n in names:
        assert getattr(lib(), n) is not None
    assert "workspace" in hkg.hkg_status_string(hkg.HKG_ERR_WORKSPACE)


def quantize(operand=0, rows=64, K=64, x=P[0], t=0, ldx=0, codes=P[1], packed=P[2]):
    return lib().hkg_mxfp4_quantize(operand, rows, K, x, t, ldx, codes, packed, None)


@pytest.mark.parametrize("kw,status", [
    (dict(operand=2), hkg.HKG_ERR_OPTS), (dict(t=2), hkg.HKG_ERR_OPTS), (dict(t=-1), hkg.HKG_ERR_OPTS),
    (dict(rows=-1), hkg.HKG_ERR_SHAPE), (dict(K=-32), hkg.HKG_ERR_SHAPE),
    (dict(x=None), hkg.HKG_ERR_NULL), (dict(codes=None), hkg.HKG_ERR_NULL), (dict(packed=None), hkg.HKG_ERR_NULL),
    (dict(ldx=63), hkg.HKG_ERR_OPTS), (dict(ldx=-1), hkg.HKG_ERR_OPTS),
    (dict(x=P[0] + 1), hkg.HKG_ERR_ALIGN), (dict(x=P[0] + 2, t=1), hkg.HKG_ERR_ALIGN),
    (dict(codes=P[1] + 8), hkg.HKG_ERR_ALIGN), (dict(packed=P[2] + 4), hkg.HKG_ERR_ALIGN),
    (dict(K=1 << 23), hkg.HKG_ERR_SIZE), (dict(K=(1 << 63) - 1), hkg.HKG_ERR_SIZE),
    (dict(rows=1 << 31), hkg.HKG_ERR_SIZE), (dict(ldx=1 << 31), hkg.HKG_ERR_SIZE),
    (dict(codes=P[0]), hkg.HKG_ERR_OVERLAP), (dict(packed=P[1] + 2032), hkg.HKG_ERR_OVERLAP),
    (dict(packed=P[0] + 64), hkg.HKG_ERR_OVERLAP),
    (dict(rows=0, x=None), hkg.HKG_OK), (dict(K=0, codes=None), hkg.HKG_OK),
])
def test_quantize_refusals(kw, status):
    assert quantize(**kw) == status


def test_quantize_both_refusals():
    f = lib().hkg_mxfp4_quantize_both
    assert f(0, 1, 64, 64, P[0], 0, 0, P[1], P[2], None, P[4], None) == hkg.HKG_ERR_NULL
    assert f(0, 3, 64, 64, P[0], 0, 0, P[1], P[2], P[3], P[4], None) == hkg.HKG_ERR_OPTS
    assert f(0, 1, 64, 64, P[0], 0, 0, P[1], P[2], P[3], P[3] + 16, None) == hkg.HKG_ERR_OVERLAP
    assert f(0, 1, 1 << 23, 64, P[0], 0, 0, P[1], P[2], P[3], P[4], None) == hkg.HKG_ERR_SIZE
    assert f(0, 1, 64, 64, P[0], 0, 0, P[1], P[2], P[3] + 4, P[4], None) == hkg.HKG_ERR_ALIGN


def test_dequantize_refusals():
    f = lib().hkg_mxfp4_dequantize
    assert f(0, 64, 64, P[0], P[1], P[2], 5, 0, None) == hkg.HKG_ERR_OPTS
    assert f(9, 64, 64, P[0], P[1], P[2], 0, 0, None) == hkg.HKG_ERR_OPTS
    assert f(0, 64, 40, P[0], P[1], P[2], 0, 48, None) == hkg.HKG_ERR_OPTS     # below the padded row
    assert f(0, 64, 64, P[0], P[1], P[0] + 16, 0, 0, None) == hkg.HKG_ERR_OVERLAP
    assert f(0, 64, 64, P[0], P[1], P[2] + 1, 0, 0, None) == hkg.HKG_ERR_ALIGN
    assert f(0, 64, 64, None, P[1], P[2], 0, 0, None) == hkg.HKG_ERR_NULL
    assert f(0, 0, 64, None, None, None, 0, 0, None) == hkg.HKG_OK


def gemm(M=64, N=64, K=64, A=P[0], B=P[1], SA=P[2], SB=P[3], C=P[4], Cf=None, ldc=0):
    return lib().hkg_gemm_mxfp4(M, N, K, A, B, SA, SB, C, Cf, ldc, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), hkg.HKG_ERR_SHAPE), (dict(K=-1), hkg.HKG_ERR_SHAPE),
    (dict(A=None), hkg.HKG_ERR_NULL), (dict(SA=None), hkg.HKG_ERR_NULL), (dict(B=None), hkg.HKG_ERR_NULL),
    (dict(SB=None), hkg.HKG_ERR_NULL), (dict(C=None), hkg.HKG_ERR_NULL),
    (dict(A=P[0] + 8), hkg.HKG_ERR_ALIGN), (dict(C=P[4] + 2), hkg.HKG_ERR_ALIGN), (dict(Cf=P[5] + 4), hkg.HKG_ERR_ALIGN),
    (dict(ldc=63), hkg.HKG_ERR_OPTS), (dict(K=1 << 23), hkg.HKG_ERR_SIZE), (dict(M=1 << 31), hkg.HKG_ERR_SIZE),
    (dict(C=P[0]), hkg.HKG_ERR_OVERLAP), (dict(Cf=P[4] + 16), hkg.HKG_ERR_OVERLAP), (dict(C=P[3] + 16), hkg.HKG_ERR_OVERLAP),
    (dict(M=0, A=None, C=None), hkg.HKG_OK), (dict(N=0, B=None), hkg.HKG_OK),
])
def test_gemm_refusals(kw, status):
    assert gemm(**kw) == status


def test_gemm_operands_may_alias():
    assert gemm(B=P[0], SB=P[2]) in (hkg.HKG_OK, hkg.HKG_ERR_DEVICE)


def linear(M=20, N=64, K=64, x=P[0], t=0, ldx=0, W=P[1], SW=P[2], y=P[3], ldy=0, ws=P[4], n=BIG):
    return lib().hkg_linear_mxfp4(M, N, K, x, t, ldx, W, SW, y, ldy, ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(t=7), hkg.HKG_ERR_OPTS), (dict(N=-1), hkg.HKG_ERR_SHAPE), (dict(x=None), hkg.HKG_ERR_NULL),
    (dict(ws=None), hkg.HKG_ERR_NULL), (dict(n=16), hkg.HKG_ERR_WORKSPACE), (dict(ws=P[4] + 4), hkg.HKG_ERR_ALIGN),
    (dict(ldx=32), hkg.HKG_ERR_OPTS), (dict(y=P[0]), hkg.HKG_ERR_OVERLAP), (dict(ws=P[1]), hkg.HKG_ERR_OVERLAP),
    (dict(ws=P[3] + 16), hkg.HKG_ERR_OVERLAP), (dict(M=0, x=None, ws=None), hkg.HKG_OK),
])
def test_linear_refusals(kw, status):
    assert linear(**kw) == status


def test_workspace_sizes():
    f, b = lib().hkg_linear_mxfp4_workspace_bytes, lib().hkg_linear_mxfp4_backward_workspace_bytes
    assert f(1, 4096, 4096) == 0                        # quantised inside the product
    assert f(20, 64, 64) >= 20 * 32 + 512
    assert f(-1, 1, 1) == hkg.HKG_ERR_SHAPE and f(64, 64, 1 << 23) == hkg.HKG_ERR_SIZE
    assert b(64, 96, 64) >= 64 * 48 + 96 * 32
    assert b(64, -1, 64) == hkg.HKG_ERR_SHAPE and b(1 << 23, 64, 64) == hkg.HKG_ERR_SIZE
    assert lib().hkg_mxfp4_code_bytes(3, 33) == 96
    assert lib().hkg_mxfp4_code_bytes(3, -1) == hkg.HKG_ERR_SHAPE
    assert lib().hkg_mxfp4_code_bytes(3, (1 << 63) - 1) == hkg.HKG_ERR_SIZE


def backward(M=64, N=64, K=64, dy=P[0], t=0, lddy=0, Wt=P[1], SWt=P[2], Xt=P[3], SXt=P[4], dx=P[5], lddx=0,
             dw=P[6], lddw=0, ws=P[7], n=BIG):
    return lib().hkg_linear_mxfp4_backward(M, N, K, dy, t, lddy, Wt, SWt, Xt, SXt, dx, lddx, dw, lddw, ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(t=7), hkg.HKG_ERR_OPTS), (dict(K=-1), hkg.HKG_ERR_SHAPE), (dict(dy=None), hkg.HKG_ERR_NULL),
    (dict(Wt=None), hkg.HKG_ERR_NULL), (dict(SXt=None), hkg.HKG_ERR_NULL), (dict(ws=None), hkg.HKG_ERR_NULL),
    (dict(n=1024), hkg.HKG_ERR_WORKSPACE), (dict(dw=P[5] + 16), hkg.HKG_ERR_OVERLAP), (dict(dx=P[0]), hkg.HKG_ERR_OVERLAP),
    (dict(ws=P[3]), hkg.HKG_ERR_OVERLAP), (dict(lddx=63), hkg.HKG_ERR_OPTS), (dict(lddy=1), hkg.HKG_ERR_OPTS),
    (dict(dx=None, dw=None), hkg.HKG_OK), (dict(K=0, dy=None, ws=None), hkg.HKG_OK),
    (dict(dx=P[5] + 8), hkg.HKG_ERR_ALIGN),
])
def test_backward_refusals(kw, status):
    assert backward(**kw) == status


def orth(rows=64, cols=96, G=P[0], t=0, ldg=0, steps=5, eps=1e-7, out=P[1], ldo=0, ws=P[2], n=BIG):
    return lib().hkg_orthogonalize(rows, cols, G, t, ldg, steps, 3.4445, -4.775, 2.0315, eps, out, ldo, ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(t=2), hkg.HKG_ERR_OPTS), (dict(steps=-1), hkg.HKG_ERR_OPTS), (dict(steps=65), hkg.HKG_ERR_OPTS),
    (dict(eps=-1.0), hkg.HKG_ERR_OPTS), (dict(eps=float("nan")), hkg.HKG_ERR_OPTS),
    (dict(rows=-1), hkg.HKG_ERR_SHAPE), (dict(G=None), hkg.HKG_ERR_NULL), (dict(out=None), hkg.HKG_ERR_NULL),
    (dict(ws=None), hkg.HKG_ERR_NULL), (dict(n=1 << 10), hkg.HKG_ERR_WORKSPACE), (dict(ws=P[2] + 8), hkg.HKG_ERR_ALIGN),
    (dict(G=P[0] + 1), hkg.HKG_ERR_ALIGN), (dict(ldg=95), hkg.HKG_ERR_OPTS), (dict(ldo=95), hkg.HKG_ERR_OPTS),
    (dict(rows=1 << 23), hkg.HKG_ERR_SIZE), (dict(cols=(1 << 63) - 1), hkg.HKG_ERR_SIZE),
    (dict(out=P[0] + 2), hkg.HKG_ERR_OVERLAP), (dict(out=P[0], t=1), hkg.HKG_ERR_OVERLAP),
    (dict(out=P[0], ldo=100), hkg.HKG_ERR_OVERLAP), (dict(ws=P[0]), hkg.HKG_ERR_OVERLAP), (dict(ws=P[1]), hkg.HKG_ERR_OVERLAP),
    (dict(rows=0, G=None, ws=None), hkg.HKG_OK),
])
def test_orthogonalize_refusals(kw, status):
    assert orth(**kw) == status


def test_orthogonalize_workspace_size():
    f = lib().hkg_orthogonalize_workspace_bytes
    assert f(64, 64) >= 5 * 64 * 64 * 2 and f(100, 30) == f(30, 100) and f(0, 5) == 0
    assert f(-1, 5) == hkg.HKG_ERR_SHAPE and f(1 << 23, 5) == hkg.HKG_ERR_SIZE
