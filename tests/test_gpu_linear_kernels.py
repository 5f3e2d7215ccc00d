"""The linear layer at the sizes where one of its kernels, or a way of dividing the work,
begins or ends: two groups of waves on odd numbers of K steps, parts of K of uneven
length, partial rounds cut by rows and by columns, transposed operands that end inside a
step, a tile or a 16-byte chunk."""
import numpy as np
import pytest

from oracle import linear as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("no GPU", allow_module_level=True)

import dense_gemm_fp8_amd as hkg  # noqa: E402

from test_gpu_linear import RNG, close, f64, normal  # noqa: E402


def some(n, k=40):
    """Rows from every part of n."""
    r = np.unique(np.r_[0:k, n // 3:n // 3 + k, n // 2:n // 2 + k, n - k:n])
    return r[(r >= 0) & (r < n)]


# two groups (12 K steps and more on at most 256 tiles): 13 and 12 steps, the last one partial;
# parts of 22, 26 and 43 steps; a grid cut by rows and one cut by columns
FORWARD = [(1024, 1100, 832), (1000, 1030, 744), (130, 4100, 4104), (260, 2100, 8200), (1000, 1030, 8200), (20, 4097, 14336),
           (4200, 4200, 72), (400, 38400, 72), (2500, 2500, 136), (70, 1030, 1032)]


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("M,N,K", FORWARD)
def test_forward(kind, M, N, K):
    x, W = normal(1, M, K, kind=kind), normal(2, N, K, size=K ** -0.5, kind=kind)
    b, at = normal(3, N, kind="fp32"), some(M)
    rows = torch.from_numpy(at).cuda()
    keep = np.concatenate([ref.keep(1, N, 0.25, RNG, int(i)) for i in at])
    for yk in (kind, "fp32"):
        r = normal(4, M, N, kind=yk)
        z = torch.empty(M, N, dtype=x.dtype, device="cuda")
        y = hkg.linear(x, W, bias=b, activation="silu", residual=r, p=0.25, rng=RNG, z=z)
        want, tol, zw, zt = ref.linear(f64(x[rows]), f64(W), f64(b), "silu", None, 0.0, None, yk, kind)
        s = ref.scale(0.25)
        want, tol = np.where(keep, want * s, 0.0), np.where(keep, tol * s, 0.0) + 2.0 ** -22 * np.abs(want) * s + ref.TINY[yk]
        v = f64(r[rows])
        want = want + v
        tol = tol + (2.0 ** -24 + ref.HALF[yk]) * (np.abs(want) + tol)
        close(y[rows], want, tol, "y %s" % yk)
        close(z[rows], zw, zt, "z")
        assert torch.equal(hkg.linear(x, W, bias=b, activation="silu", residual=r, p=0.25, rng=RNG), y)


# dx is M x K with N long, dw N x K with M long: contractions that end inside a step and an
# 8-element chunk, both small and large, parts of 68 steps (two groups), cut grids
BACKWARD = [(13000, 1100, 1032), (72, 400, 38400), (77, 4200, 4200), (1000, 4100, 264), (131, 1300, 2056), (5000, 77, 520),
            (3, 700, 1400), (700, 3, 1400), (2049, 2051, 2056)]


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("M,N,K", BACKWARD)
def test_backward(kind, M, N, K):
    x, W = normal(1, M, K, kind=kind), normal(2, N, K, size=K ** -0.5, kind=kind)
    dy, z = normal(3, M, N, size=0.5, kind=kind), normal(4, M, N, kind=kind)
    got = hkg.linear_backward(dy, x, W, z=z, activation="gelu_tanh", p=0.1, rng=RNG)
    # rows of each gradient from every part, against the oracle on what they depend on
    s, act = ref.scale(0.1), "gelu_tanh"
    keep = ref.keep(M, N, 0.1, RNG)
    dz = np.where(keep, f64(dy) * ref.slope(f64(z), act) * s, 0.0)
    e = np.where(keep, np.abs(f64(dy)) * ref.SLOPE_ERROR * s, 0.0) + 2.0 ** -22 * np.abs(dz)
    e16 = e + ref.HALF[kind] * (np.abs(dz) + e) + ref.TINY[kind]
    X, A = f64(x), f64(W)

    def product(d, off, b, n):
        w, t = d @ b, off @ np.abs(b) + (n + 1) * 2.0 ** -23 * ((np.abs(d) + off) @ np.abs(b))
        return w, t + ref.HALF[kind] * (np.abs(w) + t) + ref.TINY[kind]

    r = some(M, 24)
    close(got[0][torch.from_numpy(r).cuda()], *product(dz[r], e16[r], A, N), "dx")
    r = some(N, 24)
    close(got[1][torch.from_numpy(r).cuda()], *product(dz.T[r], e16.T[r], X, M), "dw")
    close(got[2], dz.sum(0), e.sum(0) + (M + 1) * 2.0 ** -24 * np.abs(dz).sum(0) + ref.TINY["fp32"], "dbias")
    again = hkg.linear_backward(dy, x, W, z=z, activation="gelu_tanh", p=0.1, rng=RNG)
    for a, b in zip(got, again):
        assert torch.equal(a, b)
    # each gradient alone has the same bits
    for i, kw in enumerate((dict(need_dw=False, need_dbias=False), dict(need_dx=False, need_dbias=False), dict(need_dx=False, need_dw=False))):
        assert torch.equal(hkg.linear_backward(dy, x, W, z=z, activation="gelu_tanh", p=0.1, rng=RNG, **kw)[i], got[i])


def test_what_lies_past_the_operands_is_never_read_into_a_result():
    """NaNs beside the rows and behind the last one of x, W and dy, which the products' last
    steps and tiles reach for."""
    for M, N, K in ((70, 1030, 1032), (300, 520, 136), (2100, 2304, 72), (1000, 4100, 264), (77, 4200, 520)):
        def surrounded(seed, rows, cols, pad):
            t = torch.full((rows + 70, cols + pad), float("nan"), dtype=torch.bfloat16, device="cuda")
            v = t[:rows, :cols]
            v.copy_(normal(seed, rows, cols))
            return v
        x, W, dy = surrounded(1, M, K, 24), surrounded(2, N, K, 8), surrounded(3, M, N, 13)
        assert torch.isfinite(hkg.linear(x, W)).all()
        for g in hkg.linear_backward(dy, x, W):
            assert torch.isfinite(g).all()
        want = hkg.linear_backward(dy.contiguous(), x.contiguous(), W.contiguous())
        for a, b in zip(hkg.linear_backward(dy, x, W), want):
            assert torch.equal(a, b)


def test_operands_beyond_two_gigabytes():
    """A contraction whose operand is larger than a buffer's 32-bit range."""
    M, N, K = 600_000, 40, 2048                     # x is 2.4 GB
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    x.zero_()
    x[::1000] = normal(1, M // 1000, K)
    x[-7:] = normal(2, 7, K)
    dy = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    rows = torch.cat([torch.arange(0, M, 1000), torch.arange(M - 7, M)]).cuda()
    dy[rows] = normal(3, len(rows), N)
    _, dw, db = hkg.linear_backward(dy, x, None, need_dx=False)
    d, X = f64(dy[rows]), f64(x[rows])
    w = d.T @ X
    t = (len(rows) + 1) * 2.0 ** -23 * (np.abs(d).T @ np.abs(X))
    close(dw, w, t + ref.HALF["bf16"] * (np.abs(w) + t) + ref.TINY["bf16"], "dw")
    close(db, d.sum(0), (len(rows) + 1) * 2.0 ** -24 * np.abs(d).sum(0) + ref.TINY["fp32"], "dbias")
    W = normal(4, N, K, size=K ** -0.5)
    y = hkg.linear(x, W)
    want, tol, _, _ = ref.linear(f64(x[rows]), f64(W))
    close(y[rows], want, tol, "y")


@pytest.mark.parametrize("M,N,K", [(2048, 64, 64), (1500, 72, 72), (500, 1000, 768), (1200, 1000, 776), (4100, 300, 264)])
def test_a_gradient_has_the_same_bits_whichever_others_are_asked_for(M, N, K):
    x, W, dy, z = normal(1, M, K), normal(2, N, K), normal(3, M, N), normal(4, M, N)
    def gradients(*need):
        return hkg.linear_backward(dy, x, W, z=z, activation="silu", p=0.2, rng=(3, 4), need_dx=need[0], need_dw=need[1],
                                   need_dbias=need[2])
    every = gradients(True, True, True)
    for need in ((True, True, False), (True, False, True), (False, True, True), (True, False, False), (False, True, False),
                 (False, False, True)):
        for got, want, asked in zip(gradients(*need), every, need):
            assert (got is not None) == asked
            assert got is None or torch.equal(got, want), need


def test_calls_at_once_on_two_streams_and_from_two_threads():
    """Every call has a workspace of its own: products whose K is split over workgroups, and
    gradients, side by side."""
    import threading
    sizes = ((100, 1024, 4096), (300, 520, 776))
    data = [(normal(4 * i + 1, M, K), normal(4 * i + 2, N, K), normal(4 * i + 3, M, N)) for i, (M, N, K) in enumerate(sizes)]

    def calls(x, W, dy, stream=None):
        return (hkg.linear(x, W, activation="silu", p=0.1, rng=(1, 2), stream=stream),
                *hkg.linear_backward(dy, x, W, p=0.1, rng=(1, 2), stream=stream))
    want = [calls(*d) for d in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in data]
    got = [[], []]
    for _ in range(10):
        for i in range(2):
            got[i].append(calls(*data[i], stream=streams[i]))
    torch.cuda.synchronize()
    threaded = [[], []]

    def work(i):
        for _ in range(10):
            threaded[i].append(calls(*data[i], stream=streams[i]))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for runs in (got, threaded):
        for i in range(2):
            assert len(runs[i]) == 10
            for one in runs[i]:
                for u, v in zip(one, want[i]):
                    assert torch.equal(u, v)
