"""Host side of include/hkg_linear.h on the CPU: the library exports what the header
declares, every refusal happens before any launch, and the Python functions refuse
what they cannot pass on."""
import ctypes
import os
import re

import pytest

import dense_gemm_fp8_amd as hkg
from dense_gemm_fp8_amd import linear16 as lin

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
G = 1 << 36                                  # distinct fake buffers, 64 GiB apart, never read
P = [i * G for i in range(1, 16)]
BIG = 1 << 50
OK, NULL, SHAPE, ALIGN, SIZE, OPTS, OVERLAP, SPACE = (
    hkg.HKG_OK, hkg.HKG_ERR_NULL, hkg.HKG_ERR_SHAPE, hkg.HKG_ERR_ALIGN, hkg.HKG_ERR_SIZE, hkg.HKG_ERR_OPTS,
    hkg.HKG_ERR_OVERLAP, hkg.HKG_ERR_WORKSPACE)


def lib():
    return lin._lib()


def test_library_exports_every_declared_symbol():
    text = open(os.path.join(ROOT, "include", "hkg_linear.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = re.findall(r"\b(hkg_[a-z0-9_]+)\s*\(", text)
    assert list(lin.LINEAR_EXPORTS) == names
    for n in names:
        assert getattr(lib(), n) is not None


def test_structures_have_the_c_layout():
    assert ctypes.sizeof(lin.hkg_dropout_opts) == 32 and lin.hkg_dropout_opts.seed.offset == 8
    assert ctypes.sizeof(lin.hkg_epilogue) == 80 and lin.hkg_epilogue.dropout.offset == 48


def drop(p=0.1, seed=1, offset=2, rng=None):
    return lin.hkg_dropout_opts(p, seed, offset, rng)


def dropout(rows=64, cols=64, x=P[0], t=0, ldx=0, d="default", r=None, ldr=0, out=P[1], ot=0, ldo=0):
    return lib().hkg_dropout(rows, cols, x, t, ldx, drop() if d == "default" else d, r, ldr, out, ot, ldo, None)


@pytest.mark.parametrize("kw,status", [
    (dict(t=3), OPTS), (dict(t=-1), OPTS), (dict(ot=2), OPTS), (dict(t=1, ot=0), OPTS), (dict(t=2, ot=0), OPTS),
    (dict(d=drop(p=-0.1)), OPTS), (dict(d=drop(p=1.5)), OPTS), (dict(d=drop(p=float("nan"))), OPTS),
    (dict(d=drop(rng=P[5] + 4)), ALIGN),
    (dict(rows=-1), SHAPE), (dict(cols=-1), SHAPE), (dict(x=None), NULL), (dict(out=None), NULL),
    (dict(x=P[0] + 1), ALIGN), (dict(t=1, ot=1, x=P[0] + 2), ALIGN), (dict(out=P[1] + 1), ALIGN),
    (dict(r=P[2] + 1), ALIGN), (dict(ot=1, r=P[2] + 2), ALIGN),
    (dict(ldx=63), OPTS), (dict(ldo=63), OPTS), (dict(r=P[2], ldr=63), OPTS), (dict(ldx=-64), OPTS),
    (dict(rows=1 << 31), SIZE), (dict(cols=1 << 31), SIZE), (dict(ldx=1 << 31), SIZE),
    (dict(rows=(1 << 63) - 1), SIZE), (dict(cols=(1 << 63) - 1), SIZE), (dict(ldo=(1 << 63) - 1), SIZE),
    (dict(out=P[0] + 2), OVERLAP), (dict(out=P[0], ldo=65), OVERLAP), (dict(out=P[0], ot=1), OVERLAP),
    (dict(out=P[2] + 64, r=P[2]), OVERLAP), (dict(out=P[2], r=P[2], ldo=66), OVERLAP),
    (dict(d=drop(rng=P[1] + 8)), OVERLAP),
    (dict(rows=0, x=None, out=None), OK), (dict(cols=0, x=None, out=None), OK),
])
def test_dropout_refusals(kw, status):
    assert dropout(**kw) == status


def epilogue(bias=None, bt=0, act=0, r=None, ldr=0, z=None, ldz=0, d=None):
    return lin.hkg_epilogue(bias, bt, act, r, ldr, z, ldz, d or drop(0.0))


def linear(M=64, N=64, K=64, t=0, x=P[0], ldx=0, W=P[1], ldw=0, e=None, y=P[2], yt=0, ldy=0, ws=None, n=0):
    return lib().hkg_linear(M, N, K, t, x, ldx, W, ldw, e, y, yt, ldy, ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(t=1), OPTS), (dict(t=3), OPTS), (dict(yt=2), OPTS), (dict(t=2, yt=0), OPTS), (dict(yt=9), OPTS),
    (dict(e=epilogue(act=5)), OPTS), (dict(e=epilogue(act=-1)), OPTS), (dict(e=epilogue(bias=P[3], bt=2)), OPTS),
    (dict(e=epilogue(d=drop(2.0))), OPTS), (dict(e=epilogue(d=drop(float("inf")))), OPTS),
    (dict(M=-1), SHAPE), (dict(N=-1), SHAPE), (dict(K=-8), SHAPE), (dict(K=60), SHAPE), (dict(K=(1 << 63) - 1), SHAPE),
    (dict(x=None), NULL), (dict(W=None), NULL), (dict(y=None), NULL),
    (dict(x=P[0] + 8), ALIGN), (dict(W=P[1] + 2), ALIGN), (dict(ldx=68), ALIGN), (dict(ldw=70), ALIGN),
    (dict(y=P[2] + 1), ALIGN), (dict(y=P[2] + 2, yt=1), ALIGN), (dict(e=epilogue(bias=P[3] + 1)), ALIGN),
    (dict(e=epilogue(bias=P[3] + 2, bt=1)), ALIGN), (dict(e=epilogue(r=P[3] + 1)), ALIGN),
    (dict(e=epilogue(z=P[3] + 1)), ALIGN), (dict(e=epilogue(d=drop(0.5, rng=P[3] + 4))), ALIGN),
    (dict(ldx=56), OPTS), (dict(ldw=8), OPTS), (dict(ldy=63), OPTS), (dict(e=epilogue(r=P[3], ldr=1)), OPTS),
    (dict(e=epilogue(z=P[3], ldz=63)), OPTS), (dict(ldy=-1), OPTS),
    (dict(K=1 << 22), SIZE), (dict(ldx=1 << 22), SIZE), (dict(ldw=1 << 40), SIZE), (dict(M=1 << 31), SIZE),
    (dict(N=1 << 31), SIZE), (dict(ldy=1 << 31), SIZE), (dict(ldy=(1 << 63) - 1), SIZE), (dict(K=(1 << 62)), SIZE),
    (dict(N=(1 << 63) - 1), SIZE), (dict(K=0, N=1 << 31), SIZE), (dict(M=1 << 18, N=1 << 21), SIZE),
    (dict(M=(1 << 31) - 1, N=(1 << 31) - 1, ldx=64, ldw=64), SIZE),
    (dict(y=P[0]), OVERLAP), (dict(y=P[1] + 64), OVERLAP), (dict(e=epilogue(z=P[2] + 16)), OVERLAP),
    (dict(e=epilogue(z=P[0])), OVERLAP), (dict(e=epilogue(bias=P[2] + 4)), OVERLAP),
    (dict(e=epilogue(r=P[2] + 2)), OVERLAP), (dict(e=epilogue(r=P[2], ldr=72)), OVERLAP),
    (dict(e=epilogue(r=P[3], z=P[3])), OVERLAP), (dict(e=epilogue(d=drop(0.5, rng=P[2]))), OVERLAP),
    (dict(e=epilogue(r=P[2], z=P[2] + 4096)), OVERLAP),
    (dict(M=0, x=None, y=None), OK), (dict(N=0, W=None, y=None), OK),
])
def test_linear_refusals(kw, status):
    assert linear(**kw) == status


def backward(M=64, N=64, K=64, t=0, dy=P[0], dt=0, lddy=0, x=P[1], ldx=0, W=P[2], ldw=0, z=P[3], ldz=0, act=2, d=None,
             dx=P[4], lddx=0, dw=P[5], lddw=0, db=P[6], ws=P[7], n=BIG):
    return lib().hkg_linear_backward(M, N, K, t, dy, dt, lddy, x, ldx, W, ldw, z, ldz, act, d, dx, lddx, dw, lddw, db, ws, n,
                                     None)


@pytest.mark.parametrize("kw,status", [
    (dict(t=1), OPTS), (dict(dt=2), OPTS), (dict(t=2, dt=0), OPTS), (dict(act=7), OPTS), (dict(d=drop(-1.0)), OPTS),
    (dict(M=-1), SHAPE), (dict(K=4), SHAPE), (dict(N=-5), SHAPE),
    (dict(dy=None), NULL), (dict(x=None), NULL), (dict(W=None), NULL), (dict(z=None), NULL), (dict(ws=None), NULL),
    (dict(dy=P[0] + 1), ALIGN), (dict(dy=P[0] + 2, dt=1), ALIGN), (dict(x=P[1] + 8), ALIGN), (dict(W=P[2] + 8), ALIGN),
    (dict(z=P[3] + 1), ALIGN), (dict(dx=P[4] + 1), ALIGN), (dict(db=P[6] + 2), ALIGN), (dict(ws=P[7] + 8), ALIGN),
    (dict(ldx=68), ALIGN), (dict(d=drop(0.1, rng=P[8] + 1)), ALIGN),
    (dict(lddy=63), OPTS), (dict(ldx=56), OPTS), (dict(ldw=56), OPTS), (dict(ldz=63), OPTS), (dict(lddx=63), OPTS),
    (dict(lddw=63), OPTS),
    (dict(M=1 << 22), SIZE), (dict(N=1 << 22), SIZE), (dict(K=1 << 22), SIZE), (dict(M=(1 << 63) - 1), SIZE),
    (dict(M=1 << 21, N=1 << 21), SIZE), (dict(lddy=1 << 31), SIZE), (dict(lddw=(1 << 63) - 1), SIZE),
    (dict(n=1024), SPACE), (dict(dx=P[5] + 16), OVERLAP), (dict(dw=P[0]), OVERLAP), (dict(dx=P[2]), OVERLAP),
    (dict(db=P[4] + 16), OVERLAP), (dict(ws=P[1]), OVERLAP), (dict(ws=P[4] - 16), OVERLAP), (dict(db=P[3]), OVERLAP),
    (dict(d=drop(0.1, rng=P[6])), OVERLAP),
    (dict(dx=None, dw=None, db=None), OK), (dict(K=0, db=None, dy=None), OK), (dict(N=0, M=0), OK),
])
def test_backward_refusals(kw, status):
    assert backward(**kw) == status


def test_workspace_sizes():
    f, b = lib().hkg_linear_workspace_bytes, lib().hkg_linear_backward_workspace_bytes
    assert f(1, 4096, 4096) >= 0 and f(-1, 1, 8) == SHAPE and f(1, 1, 4) == SHAPE and f(1, 1, 1 << 22) == SIZE
    assert f(1 << 31, 1, 8) == SIZE
    assert b(64, 96, 64) > 0 and b(64, -1, 64) == SHAPE and b(64, 64, 1 << 22) == SIZE and b(1 << 22, 64, 64) == SIZE
    for m in (0, 1, 3000):
        for n in (0, 1, 3000):
            for k in (0, 8, 2048):
                assert f(m, n, k) >= 0 and b(m, n, k) >= 0


def test_python_refusals():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        hkg.linear(x, x)                                   # not on a GPU
    with pytest.raises(TypeError):
        hkg.linear(x.float(), x)
    with pytest.raises(TypeError):
        hkg.dropout(x.int(), 0.1, (0, 0))
    with pytest.raises(ValueError):
        hkg.dropout(x, 0.1, (0, 0))
    with pytest.raises(ValueError):
        hkg.linear_backward(x, None, None)
    opts = lin.hkg_dropout_opts()
    for p, rng in ((-0.1, (0, 0)), (1.1, (0, 0)), (float("nan"), (0, 0)), (0.1, None), (0.1, (-1, 0)), (0.1, (0, 1 << 64)),
                   (0.1, torch.zeros(2)), (0.1, torch.zeros(3, dtype=torch.int64)), (0.1, torch.zeros(2, dtype=torch.int64))):
        with pytest.raises(ValueError):
            lin._dropout(opts, p, rng)
    with pytest.raises(ValueError):
        lin._activation("swish")
    assert lin._dropout(opts, 0.0, None) is None and lin._dropout(opts, 0.5, ((1 << 64) - 1, 3)) is None
    assert opts.seed == (1 << 64) - 1 and opts.offset == 3
