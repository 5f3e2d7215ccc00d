"""GPU tests of hkg_orthogonalize (include/hkg_ops.h) against its iteration in
numpy and 64 bits.

The tolerance follows the roundings.  With u = 2^-11 (fp16, half a step, relative)
a step rounds A = X X^T, P = b A + c A A and the new X, each entry by at most u of
itself: dX' <= (|b| + 2 |c| |A|_2) u |A|_F |X|_2 + u |P|_F |X|_2 + u |X'|_F, and an
error in X passes on by at most L = max(|p'|, |p(s)/s|) over the singular values s.
Entrywise roundings are independent, so their squares add, with u / sqrt(3) each; the
test allows three times that, plus the bf16 rounding of the result (2^-8)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("no GPU", allow_module_level=True)

import dense_gemm_fp8_amd as hkg  # noqa: E402
from dense_gemm_fp8_amd import ops  # noqa: E402

COEFFS, EPS = (3.4445, -4.7750, 2.0315), 1e-7


def host(t):
    torch.cuda.synchronize()
    return t.float().cpu().numpy().astype(np.float64)


def reference(G, steps=5, coeffs=COEFFS, eps=EPS):
    """(X after `steps`, tolerance of its Frobenius norm)."""
    a, b, c = coeffs
    G = np.asarray(G, dtype=np.float64)
    tall = G.shape[0] > G.shape[1]
    X = (G.T if tall else G) / (np.linalg.norm(G) + eps)
    m, n = X.shape
    u, fro = 2.0 ** -11 / np.sqrt(3), np.linalg.norm
    tiny = 2.0 ** -25 / 4096.0                      # half a subnormal step, scaled
    err = u * fro(X) + tiny * np.sqrt(m * n)
    for _ in range(steps):
        A = X @ X.T
        P = b * A + c * (A @ A)
        s = np.linalg.norm(X, 2)
        grid = np.linspace(0, s, 200)
        L = max(np.abs(a + 3 * b * grid ** 2 + 5 * c * grid ** 4).max(), np.abs(a + b * grid ** 2 + c * grid ** 4).max())
        new = a * X + P @ X
        d = [u * fro(A) * (abs(b) + 2 * abs(c) * s * s) * s, u * fro(P) * s, u * fro(new), tiny * np.sqrt(m * n) * 4]
        err = np.sqrt((L * err) ** 2 + sum(v * v for v in d))
        X = new
    return (X.T if tall else X), 3 * err + 2.0 ** -8 * fro(X)


def gradient(seed, rows, cols, dtype=torch.float32, scale=1e-3):
    g = torch.Generator().manual_seed(seed)
    r = min(4, rows, cols)
    x = torch.randn(rows, r, generator=g) @ torch.randn(r, cols, generator=g) + torch.randn(rows, cols, generator=g)
    return (scale * x).to(dtype)


def check(out, G, **kw):
    want, tol = reference(G.double().numpy(), **kw)
    got = host(out)
    off = np.linalg.norm(got - want)
    assert np.isfinite(got).all() and off <= tol, "%g off, %g allowed, of %g" % (off, tol, np.linalg.norm(want))
    # no entry, tile or edge may hide behind the norm: entries are within the
    # norm's error spread evenly, times 8 for the largest of them, and bf16's step
    each = 8 * tol / np.sqrt(want.size) + 2.0 ** -8 * np.abs(want)
    assert (np.abs(got - want) <= np.maximum(each, tol if want.size < 64 else 0)).all()


SIZES = [(1, 1), (1, 100), (100, 1), (5, 7), (64, 64), (65, 130), (130, 65), (128, 1000), (200, 200), (257, 300),
         (300, 257), (520, 1100), (1100, 520), (1300, 1300)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_five_steps(rows, cols, dtype):
    print("orth %dx%d %s" % (rows, cols, dtype), flush=True)
    G = gradient(rows + cols, rows, cols, dtype)
    check(hkg.orthogonalize(G.cuda()), G)


@pytest.mark.parametrize("steps", [0, 1, 2, 3, 8])
@pytest.mark.parametrize("rows,cols", [(96, 200), (200, 96)])
def test_other_step_counts(rows, cols, steps):
    G = gradient(steps, rows, cols)
    check(hkg.orthogonalize(G.cuda(), steps=steps), G, steps=steps)


def test_other_coefficients_converge():
    # the cubic Newton-Schulz step (3/2, -1/2, 0): singular values towards 1
    G = gradient(3, 100, 300)
    co = (1.5, -0.5, 0.0)
    out = hkg.orthogonalize(G.cuda(), steps=20, coefficients=co)
    check(out, G, steps=20, coeffs=co)


def test_transposed_input_gives_the_transposed_result():
    G = gradient(5, 150, 333)
    a = hkg.orthogonalize(G.cuda())
    b = hkg.orthogonalize(G.t().contiguous().cuda())
    assert torch.equal(a, b.t())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_views_and_in_place(dtype):
    big = gradient(6, 130, 300, dtype).cuda()
    for r, c0, c1 in ((130, 0, 296), (77, 1, 202), (129, 3, 36)):
        v = big[:r, c0:c1]
        out = torch.full((r + 1, c1 - c0 + 5), 9.0, dtype=torch.bfloat16, device="cuda")
        o = out[:r, 1:c1 - c0 + 1]
        hkg.orthogonalize(v, out=o)
        check(o, v.cpu())
        assert (host(out[r:]) == 9).all() and (host(out[:, c1 - c0 + 1:]) == 9).all() and (host(out[:, :1]) == 9).all()
    if dtype == torch.bfloat16:
        for steps in (0, 5):
            want = hkg.orthogonalize(big, steps=steps)
            mine = big.clone()
            assert hkg.orthogonalize(mine, steps=steps, out=mine) is mine
            assert torch.equal(mine, want)


def test_the_workspace_may_hold_anything():
    G = gradient(7, 140, 210).cuda()
    need = ops._lib().hkg_orthogonalize_workspace_bytes(140, 210)
    want = hkg.orthogonalize(G)
    for fill in (0, 0x7e, 0xff):
        ws = torch.full((need + 64,), fill, dtype=torch.uint8, device="cuda")
        assert torch.equal(hkg.orthogonalize(G, workspace=ws[:need]), want)
        assert (ws[need:] == fill).all()


def test_zero_tiny_huge_and_bad_values():
    z = torch.zeros(70, 90, device="cuda")
    for eps in (0.0, 1e-7):
        assert (host(hkg.orthogonalize(z, eps=eps)) == 0).all()
    assert (host(hkg.orthogonalize(z, steps=0)) == 0).all()
    for scale in (1e-30, 1e25):                     # |G|^2 leaves fp32's range
        G = gradient(8, 70, 90, scale=scale)
        check(hkg.orthogonalize(G.cuda(), eps=0.0), G, eps=0.0)
    for bad in (float("nan"), float("inf"), float("-inf")):
        G = gradient(8, 70, 90)
        G[69, 3] = bad
        assert torch.isnan(hkg.orthogonalize(G.cuda())).all()


def test_another_stream_and_graph_replays():
    G = gradient(9, 200, 320).cuda()
    want = hkg.orthogonalize(G)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = [hkg.orthogonalize(G, stream=s) for _ in range(6)]
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(o, want) for o in outs)
    with torch.cuda.stream(s):
        hkg.orthogonalize(G)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = hkg.orthogonalize(G)
    for i in range(4):
        G.copy_(gradient(20 + i, 200, 320))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, hkg.orthogonalize(G))


@pytest.mark.parametrize("rows,cols", [(1500, 1600), (2304, 2600), (2700, 2400), (4096, 14336), (6400, 5888)])
def test_every_tile_size_and_the_triangle(rows, cols):
    """Sizes that take 128-, 192- and 256-wide tiles, and whose update is split into two
    launches by columns (4096 x 14336) and by rows (6400 x 5888); checked against
    the iteration in fp64 on the GPU's own matmul."""
    G = gradient(31, rows, cols).cuda()
    X = G.double().t() if rows > cols else G.double()
    X = X / (torch.linalg.norm(X) + EPS)
    a, b, c = COEFFS
    for _ in range(5):
        A = X @ X.t()
        X = a * X + (b * A + c * (A @ A)) @ X
    X = X.t() if rows > cols else X
    got = hkg.orthogonalize(G).double()
    d = (got - X).abs()
    # the same error budget as above, at its size for these: 3 % of the largest entry
    # would already be a wrong tile; roundings stay near 1 % of the norm
    assert d.norm() <= 0.01 * X.norm()
    tiles = d[:rows // 64 * 64, :cols // 64 * 64].reshape(rows // 64, 64, cols // 64, 64).norm(dim=(1, 3))
    assert tiles.max() <= 0.03 * X.norm() / (rows * cols / 4096) ** 0.5


def reference_pairs(G, steps, coeffs=COEFFS, eps=EPS):
    """(X after `steps` in 64 bits, tolerance of its Frobenius norm).  The roundings'
    size is what they do in 64 bits with every intermediate of a pair of steps (A, P,
    B = P A, A' = P B, P', P' P and X, X times 2^12) rounded to fp16; the operator's
    differ from those in single units by the order of its sums, so it may be off by four
    times as much, plus the bf16 rounding of the result."""
    a, b, c = coeffs
    G = np.asarray(G, dtype=np.float64)
    tall = G.shape[0] > G.shape[1]
    X = (G.T if tall else G) / (np.linalg.norm(G) + eps)
    eye = np.eye(X.shape[0])

    def fp16(M, scale=1.0):
        return (M * scale).astype(np.float16).astype(np.float64) / scale

    Y, left = fp16(X, 4096.0), steps
    for _ in range(steps):
        A = X @ X.T
        X = (a * eye + b * A + c * (A @ A)) @ X
    while left:
        A = fp16(Y @ Y.T)
        Q = fp16(a * eye + b * A + c * (A @ A))
        if left >= 2:
            A2 = fp16(Q @ fp16(Q @ A))
            Q = fp16(fp16(a * eye + b * A2 + c * (A2 @ A2)) @ Q)
        Y = fp16(Q @ Y, 4096.0)
        left -= min(left, 2)
    tol = 4 * np.linalg.norm(Y - X) + 2.0 ** -8 * np.linalg.norm(X)
    return (X.T if tall else X), tol


def check_pairs(out, G, **kw):
    want, tol = reference_pairs(G.double().numpy(), **kw)
    got = host(out)
    off = np.linalg.norm(got - want)
    assert np.isfinite(got).all() and off <= tol, "%g off, %g allowed, of %g" % (off, tol, np.linalg.norm(want))
    each = 8 * tol / np.sqrt(want.size) + 2.0 ** -8 * np.abs(want)
    assert (np.abs(got - want) <= each).all()


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 5, 8])
@pytest.mark.parametrize("rows,cols", [(700, 4500), (4500, 701)])
def test_steps_in_pairs(rows, cols, steps):
    print("orth pairs %dx%d %d" % (rows, cols, steps), flush=True)
    G = gradient(7 * steps, rows, cols)
    check_pairs(hkg.orthogonalize(G.cuda(), steps=steps), G, steps=steps)


@pytest.mark.parametrize("rows,cols", [(1500, 2250), (1500, 2249), (2249, 1500), (2250, 1500), (130, 18000)])
def test_steps_in_pairs_from_where_they_start(rows, cols):
    G = gradient(8, rows, cols, torch.bfloat16)
    check_pairs(hkg.orthogonalize(G.cuda()), G, steps=5)


@pytest.mark.parametrize("coeffs,steps", [((4.0, -6.0, 2.5), 3), ((4.5, -6.0, 2.0), 2), ((-3.0, 4.0, -1.5), 4), ((1.5, -0.5, 0.0), 20)])
def test_steps_in_pairs_other_coefficients(coeffs, steps):
    """a = 4.5 takes single steps, whose error budget is below that of pairs."""
    G = gradient(9, 640, 4500)
    check_pairs(hkg.orthogonalize(G.cuda(), steps=steps, coefficients=coeffs), G, steps=steps, coeffs=coeffs)


def test_steps_in_pairs_with_small_singular_values():
    # singular values from 1 to 1e-4: those of the result, by the step's own polynomial
    g = torch.Generator().manual_seed(10)
    U = torch.linalg.qr(torch.randn(640, 640, generator=g, dtype=torch.float64))[0]
    V = torch.linalg.qr(torch.randn(4500, 640, generator=g, dtype=torch.float64))[0]
    G = ((U * torch.logspace(0, -4, 640, dtype=torch.float64)) @ V.t()).float()
    s = torch.linalg.svdvals(G.double())
    s = s / s.norm()
    for _ in range(5):
        s = COEFFS[0] * s + COEFFS[1] * s ** 3 + COEFFS[2] * s ** 5
    got = torch.diagonal(U.t() @ hkg.orthogonalize(G.cuda()).cpu().double() @ V)
    check_pairs(hkg.orthogonalize(G.cuda()), G, steps=5)
    assert (got - s).abs().max() <= 0.05


def test_steps_in_pairs_repeat_and_ignore_their_workspace():
    G = gradient(11, 700, 4500).cuda()
    need = ops._lib().hkg_orthogonalize_workspace_bytes(700, 4500)
    want = hkg.orthogonalize(G)
    for fill in (0, 0x7C, 0xFF):
        ws = torch.full((need + 512,), fill, dtype=torch.uint8, device="cuda")
        assert torch.equal(hkg.orthogonalize(G, workspace=ws[:need]), want)
        assert (ws[need:] == fill).all()
