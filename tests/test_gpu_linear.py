"""GPU tests of the 16-bit linear layer with its epilogue, its gradients and dropout
(include/hkg_linear.h) against the definitions in numpy and 64 bits
(oracle/linear.py), whose tolerances follow from the number formats."""
import numpy as np
import pytest

from oracle import linear as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("no GPU", allow_module_level=True)

import dense_gemm_fp8_amd as hkg  # noqa: E402

TYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
RNG = (0x299F31D0A4093822, 0x0370734413198A2E)


def normal(seed, *shape, size=1.0, kind="bf16"):
    g = np.random.Generator(np.random.PCG64(seed))
    return torch.from_numpy((size * g.standard_normal(shape)).astype(np.float32)).to(TYPE[kind]).cuda()


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def close(got, want, tol, what):
    got = f64(got)
    assert got.shape == want.shape, what
    fine = np.isfinite(want)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want), err_msg=what)
    bad = ~fine & ~np.isnan(want)
    np.testing.assert_array_equal(got[bad], want[bad], err_msg=what)
    with np.errstate(invalid="ignore"):
        off = np.where(fine, np.abs(got - want) - tol, -1.0)
    at = np.unravel_index(np.argmax(off), off.shape) if off.size else None
    assert not off.size or off.max() <= 0, "%s: at %s got %r want %r tolerance %r, %d of %d out" % (
        what, at, got[at], want[at], np.broadcast_to(tol, off.shape)[at], (off > 0).sum(), off.size)


# ---- the forward product --------------------------------------------------------------

# M, N, K: one row and one block, ends of blocks and tiles, odd columns, single K units,
# partial K steps; sizes that take small and large tiles, alone and in two launches
SHAPES = [(1, 1, 8), (1, 33, 64), (3, 31, 8), (16, 32, 72), (17, 65, 136), (64, 64, 64), (65, 257, 264), (130, 129, 1000),
          (256, 384, 520), (300, 520, 128), (1111, 277, 1184), (513, 2050, 200), (2100, 2304, 72), (1000, 1100, 64),
          (4200, 4100, 136), (2304, 2304, 24)]
FORMS = [  # bias, activation, residual, p, z
    (None, None, None, 0.0, False),
    ("fp32", "silu", None, 0.0, True),
    ("same", "gelu", "same", 0.1, True),
    (None, "gelu_tanh", "fp32", 0.5, False),
    ("same", "relu", "fp32", 0.0, False),
    ("fp32", None, "same", 0.25, False),
]


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_linear(kind, shape):
    M, N, K = shape
    big = M * N > 1 << 20
    forms = [FORMS[(SHAPES.index(shape) + (kind == "fp16")) % len(FORMS)], FORMS[2]] if big else FORMS
    x, W = normal(1, M, K, kind=kind), normal(2, N, K, size=K ** -0.5, kind=kind)
    for bias, act, residual, p, with_z in forms:
        b = None if bias is None else normal(3, N, kind=kind if bias == "same" else "fp32")
        r = None if residual is None else normal(4, M, N, kind=kind if residual == "same" else "fp32")
        z = torch.full((M, N), 7.0, dtype=TYPE[kind], device="cuda") if with_z else None
        y = hkg.linear(x, W, bias=b, activation=act, residual=r, p=p, rng=RNG, z=z)
        y_type = kind if residual != "fp32" else "fp32"
        assert y.dtype is TYPE[y_type]
        # whole results up to a million entries, above that rows from every part
        rows = np.unique(np.r_[0:17, M // 2 - 9:M // 2 + 9, M - 140:M]) if big else np.arange(M)
        rows = rows[(rows >= 0) & (rows < M)]
        at = torch.from_numpy(rows).cuda()
        keep = None
        if p:
            keep = np.concatenate([ref.keep(1, N, p, RNG, int(i)) for i in rows])
        want, tol, zw, zt = ref.linear(f64(x[at]), f64(W), f64(b), act, None, 0.0, None, y_type, kind)
        if p:   # the mask row by row, then the residual, as ref.linear does for whole matrices
            s = ref.scale(p)
            want, tol = np.where(keep, want * s, 0.0), np.where(keep, tol * s, 0.0) + 2.0 ** -22 * np.abs(want) * s + ref.TINY[y_type]
        if r is not None:
            v = f64(r[at])
            want = want + v
            tol = tol + (2.0 ** -24 + ref.HALF[y_type]) * (np.abs(want) + tol)
        close(y[at], want, tol, "y %s %s %s" % (kind, shape, (bias, act, residual, p)))
        if with_z:
            close(z[at], zw, zt, "z %s %s" % (kind, shape))


def test_small_whole_forms_agree_with_the_definition():
    """ref.linear with everything at once, as one call (the loop above applies its parts)."""
    x, W, b, r = normal(1, 37, 72), normal(2, 41, 72, size=0.1), normal(3, 41), normal(4, 37, 41)
    y = hkg.linear(x, W, bias=b, activation="gelu", residual=r, p=0.3, rng=RNG)
    want, tol, _, _ = ref.linear(f64(x), f64(W), f64(b), "gelu", f64(r), 0.3, RNG)
    close(y, want, tol, "y")


@pytest.mark.parametrize("M,N,K", [(5, 40, 72), (300, 333, 264), (2100, 2304, 72)])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_pitches_and_odd_addresses(kind, M, N, K):
    """Every matrix a view of a wider one, rows at odd addresses; what is beside them stays."""
    def wide(seed, rows, cols, at, kind):
        t = normal(seed, rows, cols + at + 9, kind=kind)
        return t, t[:, at:at + cols]

    x = normal(1, M, K + 24, kind=kind)[:, 8:8 + K]
    W = normal(2, N, K + 16, size=K ** -0.5, kind=kind)[:, 16:]
    b = normal(3, N + 1, kind=kind)[1:]
    for yk in (kind, "fp32"):
        _, r = wide(4, M, N, 3, yk)
        yw, y = wide(5, M, N, 1, yk)
        zw, z = wide(6, M, N, 5, kind)
        before, zbefore = yw.clone(), zw.clone()
        hkg.linear(x, W, bias=b, activation="gelu_tanh", residual=r, p=0.2, rng=RNG, y=y, z=z)
        plain = torch.empty_like(z.contiguous())
        want = hkg.linear(x.contiguous(), W.contiguous(), bias=b.clone(), activation="gelu_tanh", residual=r.contiguous(),
                          p=0.2, rng=RNG, z=plain)
        assert torch.equal(y, want) and torch.equal(z, plain)
        y.copy_(before[:, 1:1 + N])
        z.copy_(zbefore[:, 5:5 + N])
        assert torch.equal(yw, before) and torch.equal(zw, zbefore)


@pytest.mark.parametrize("M,N,K", [(4, 48, 64), (130, 129, 72), (2100, 2304, 64)])
def test_onto_the_residual_itself(M, N, K):
    x, W, b = normal(1, M, K), normal(2, N, K), normal(3, N)
    for yk in ("bf16", "fp32"):
        r = normal(4, M, N, kind=yk)
        want = hkg.linear(x, W, bias=b, activation="silu", residual=r, p=0.1, rng=RNG)
        got = hkg.linear(x, W, bias=b, activation="silu", residual=r, p=0.1, rng=RNG, y=r)
        assert got is r and torch.equal(r, want)


@pytest.mark.parametrize("M,N", [(1, 1), (70, 33), (300, 2000)])
def test_without_k(M, N):
    b, r = normal(3, N), normal(4, M, N)
    x, W = torch.empty(M, 0, dtype=torch.bfloat16, device="cuda"), torch.empty(N, 0, dtype=torch.bfloat16, device="cuda")
    y = hkg.linear(x, W, bias=b, activation="gelu", residual=r)
    want, tol, _, _ = ref.linear(f64(x), f64(W), f64(b), "gelu", f64(r))
    close(y, want, tol, "y")
    assert not hkg.linear(x, W).any()


def test_empty():
    x, W = normal(1, 0, 64), normal(2, 5, 64)
    assert hkg.linear(x, W).shape == (0, 5) and hkg.linear(W, x).shape == (5, 0)
    dy = normal(3, 0, 5)
    dx, dw, db = hkg.linear_backward(dy, x, W)
    assert dx.shape == (0, 64) and not dw.any() and not db.any() and dw.shape == (5, 64)
    dx, dw, db = hkg.linear_backward(dy.t().contiguous(), W, x)
    assert dx.shape == (5, 64) and not dx.any() and dw.shape == (0, 64) and db.shape == (0,)
    assert hkg.dropout(dy, 0.5, RNG).shape == (0, 5)


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_activations_over_their_range(act):
    """z is the bias: 4096 values from -40 to 40 and the ends, y in fp32."""
    z = torch.linspace(-40, 40, 4096, dtype=torch.float32)
    z[:10] = torch.tensor([float("-inf"), float("inf"), float("nan"), -3.4e38, 3.4e38, 0.0, -0.0, 1e-38, -1e30, 1e30])
    x, W = torch.zeros(1, 8, dtype=torch.bfloat16, device="cuda"), torch.zeros(4096, 8, dtype=torch.bfloat16, device="cuda")
    y = torch.empty(1, 4096, dtype=torch.float32, device="cuda")
    hkg.linear(x, W, bias=z.cuda(), activation=act, y=y)
    want = ref.act(f64(z)[None], act)
    close(y, want, ref.act_error(f64(z)[None], act) + 2.0 ** -23 * np.abs(np.where(np.isfinite(want), want, 0.0)), act)


def test_infinities_and_nans_reach_their_results_only():
    for M, N, K in ((20, 40, 64), (300, 700, 64), (2100, 2304, 64)):
        x, W = normal(1, M, K), normal(2, N, K)
        x[7, 3] = float("inf")
        W[5, 9] = float("nan")
        y = f64(hkg.linear(x, W))
        assert np.isnan(y[:, 5]).all()
        assert np.isinf(np.delete(y[7], 5)).all()
        rest = np.delete(np.delete(y, 7, 0), 5, 1)
        assert np.isfinite(rest).all()


def test_dropped_elements_are_zero_whatever_they_were():
    for M, N, K in ((20, 40, 64), (2100, 2304, 64)):
        x, W, b = normal(1, M, K), normal(2, N, K), normal(3, N, kind="fp32")
        b[::3] = float("nan")
        b[1::3] = float("inf")
        y = f64(hkg.linear(x, W, bias=b, p=0.5, rng=RNG))
        keep = ref.keep(M, N, 0.5, RNG)
        assert (y[~keep] == 0).all() and np.isnan(y[:, ::3][keep[:, ::3]]).all() and np.isinf(y[:, 1::3][keep[:, 1::3]]).all()
        dy, z = normal(4, M, N), normal(5, M, N)
        dy[0], z[1], dy[2] = float("nan"), float("nan"), float("inf")
        _, _, db = hkg.linear_backward(dy, x, W, z=z, activation="gelu", p=0.5, rng=RNG, need_dx=False, need_dw=False)
        dead = ~keep[:3].any(0)
        fine = np.isfinite(f64(db))
        np.testing.assert_array_equal(fine, dead)   # a finite sum: no bad element was kept
        v = f64(hkg.dropout(dy, 0.5, RNG))
        assert (v[~keep] == 0).all() and np.isnan(v[0][keep[0]]).all() and np.isinf(v[2][keep[2]]).all()


def test_fp16_results_beyond_its_range_are_infinities():
    x = torch.full((40, 64), 100.0, dtype=torch.float16, device="cuda")
    W = torch.full((64, 64), 100.0, dtype=torch.float16, device="cuda")
    assert torch.isinf(hkg.linear(x, W)).all()
    y = torch.empty(40, 64, dtype=torch.float32, device="cuda")
    assert (hkg.linear(x, W, y=y) == 640000.0).all()


# ---- dropout ----------------------------------------------------------------------------

@pytest.mark.parametrize("kind,out", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 9), (3, 8), (7, 77), (33, 256), (5, 2049), (1000, 17), (2, 70001), (513, 1000)])
def test_dropout(kind, out, rows, cols):
    x, r = normal(1, rows, cols, kind=kind), normal(2, rows, cols, kind=out)
    for p in (0.0, 0.1, 0.5, 1.0, 1e-6, 0.99999):
        o = torch.empty(rows, cols, dtype=TYPE[out], device="cuda")
        close(hkg.dropout(x, p, RNG, out=o), *ref.dropout(f64(x), p, RNG, None, out), "out p %g" % p)
        close(hkg.dropout(x, p, RNG, residual=r), *ref.dropout(f64(x), p, RNG, f64(r), out), "with residual p %g" % p)


def test_dropout_in_place_and_views():
    w = normal(1, 300, 140)
    x, before = w[:, 5:105], w.clone()
    want = hkg.dropout(x.contiguous(), 0.3, RNG)
    assert torch.equal(hkg.dropout(x, 0.3, RNG, out=x), want) and torch.equal(x, want)
    x.copy_(before[:, 5:105])
    assert torch.equal(w, before)
    r = normal(2, 300, 100)
    want = hkg.dropout(x, 0.3, RNG, residual=r)
    assert torch.equal(hkg.dropout(x, 0.3, RNG, residual=r, out=r), want)
    x2 = normal(3, 300, 100)
    want = hkg.dropout(x2, 0.3, RNG, residual=x2)              # x and residual may be one matrix
    assert torch.equal(hkg.dropout(x2, 0.3, RNG, residual=x2, out=x2), want)


def test_one_mask_for_every_operator():
    """The same elements fall out of dropout, linear (few rows and tiles) and the backward pass."""
    for M, N in ((10, 333), (2100, 2304)):
        keep = ref.keep(M, N, 0.25, RNG)
        ones = torch.ones(M, N, dtype=torch.bfloat16, device="cuda")
        x, W = torch.zeros(M, 8, dtype=torch.bfloat16, device="cuda"), torch.zeros(N, 8, dtype=torch.bfloat16, device="cuda")
        b = torch.ones(N, device="cuda")
        np.testing.assert_array_equal(f64(hkg.dropout(ones, 0.25, RNG)) != 0, keep)
        np.testing.assert_array_equal(f64(hkg.linear(x, W, bias=b, p=0.25, rng=RNG)) != 0, keep)
        _, _, db = hkg.linear_backward(ones, x, W, p=0.25, rng=RNG)
        # positive terms: each of at most M - 1 additions in fp32 is within 2^-24 of its
        # result, which is part of the sum, and 4 / 3 and its product round by as much
        np.testing.assert_allclose(f64(db), keep.sum(0) * (4.0 / 3.0), rtol=(M + 1) * 2.0 ** -24)


def test_rng_on_the_gpu_is_read_when_the_kernels_run():
    x = normal(1, 64, 96)
    t = torch.tensor([5, 6], dtype=torch.int64, device="cuda")
    assert torch.equal(hkg.dropout(x, 0.5, t), hkg.dropout(x, 0.5, (5, 6)))
    t[1] = 7
    assert torch.equal(hkg.dropout(x, 0.5, t), hkg.dropout(x, 0.5, (5, 7)))
    big = torch.tensor([-1, -(1 << 63)], dtype=torch.int64, device="cuda")
    assert torch.equal(hkg.dropout(x, 0.5, big), hkg.dropout(x, 0.5, ((1 << 64) - 1, 1 << 63)))


# ---- gradients ----------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 8), (5, 33, 64), (64, 64, 64), (65, 130, 72), (200, 77, 264), (129, 300, 520),
                                   (500, 1000, 768), (1030, 260, 136)])
def test_backward(kind, M, N, K):
    x, W = normal(1, M, K, kind=kind), normal(2, N, K, size=K ** -0.5, kind=kind)
    z = normal(4, M, N, size=2.0, kind=kind)
    for act, p, dk in (("gelu", 0.1, kind), (None, 0.0, "fp32"), ("silu", 0.0, "fp32"), ("relu", 0.5, kind),
                       ("gelu_tanh", 0.0, kind), (None, 0.0, kind), (None, 0.3, kind)):
        dy = normal(3, M, N, kind=dk)
        got = hkg.linear_backward(dy, x, W, z=z if act else None, activation=act, p=p, rng=RNG)
        want = ref.backward(f64(dy), f64(x), f64(W), f64(z), act, p, RNG, kind)
        for name, g, (w, tol) in zip(("dx", "dw", "dbias"), got, want):
            close(g, w, tol, "%s %s %s" % (name, kind, (M, N, K, act, p, dk)))
        one = hkg.linear_backward(dy, x, None, z=z if act else None, activation=act, p=p, rng=RNG, need_dx=False)
        assert one[0] is None and torch.equal(one[1], got[1]) and torch.equal(one[2], got[2])
        two = hkg.linear_backward(dy, None, W, z=z if act else None, activation=act, p=p, rng=RNG, need_dw=False, need_dbias=False)
        assert two[1] is None and two[2] is None and torch.equal(two[0], got[0])


@pytest.mark.parametrize("M,N,K", [(2100, 2304, 72), (600, 4160, 2048), (2304, 200, 2304)])
def test_backward_of_large_products(M, N, K):
    """Sizes that take tiles; compared in rows and columns from every part."""
    x, W, dy, z = normal(1, M, K), normal(2, N, K, size=K ** -0.5), normal(3, M, N), normal(4, M, N)
    dx, dw, db = hkg.linear_backward(dy, x, W, z=z, activation="silu")
    (wx, tx), (ww, tw), (wb, tb) = ref.backward(f64(dy), f64(x), f64(W), f64(z), "silu")
    close(dx, wx, tx, "dx")
    close(dw, ww, tw, "dw")
    close(db, wb, tb, "dbias")


def test_backward_with_views_and_outputs():
    M, N, K = 150, 140, 72
    def inside(seed, rows, cols, at, kind="bf16"):
        return normal(seed, rows, cols + 16 + at, kind=kind)[:, at:at + cols]
    x, W = inside(1, M, K, 8), inside(2, N, K, 16)
    dy, z = inside(3, M, N, 3, "fp32"), inside(4, M, N, 5)
    want = hkg.linear_backward(dy.contiguous(), x.contiguous(), W.contiguous(), z=z.contiguous(), activation="gelu", p=0.1, rng=RNG)
    dxw, dww = normal(5, M, K + 7), normal(6, N, K + 7)
    b1, b2 = dxw.clone(), dww.clone()
    db = torch.empty(N, device="cuda")
    got = hkg.linear_backward(dy, x, W, z=z, activation="gelu", p=0.1, rng=RNG, dx=dxw[:, 3:3 + K], dw=dww[:, 1:1 + K], dbias=db)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert got[2] is db
    dxw[:, 3:3 + K], dww[:, 1:1 + K] = b1[:, 3:3 + K], b2[:, 1:1 + K]
    assert torch.equal(dxw, b1) and torch.equal(dww, b2)


def test_gradients_against_differences():
    """d sum(g y) / d b, x and W of the forward pass in fp32 against linear_backward.  Inputs
    on a grid of 2^-4, so that steps of h = 2^-4 are exact in bf16; central differences are
    off by h^2 / 6 times the third derivative along the step (of silu at most 0.15 |step|^3,
    |step| <= 4 for x and W) and by y's rounding, 2^-23 |g y| summed, over h."""
    M, N, K, h = 6, 40, 16, 2.0 ** -4
    grid = lambda s, *n: (normal(s, *n, kind="fp32").clamp(-3.9, 3.9) * 16).round() / 16  # noqa: E731
    x, W, b = grid(1, M, K), grid(2, N, K) / 4, grid(3, N)
    W = (W * 16).round() / 16
    g = grid(4, M, N)
    y0 = torch.empty(M, N, device="cuda")
    z = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")

    def loss(x, W, b):
        hkg.linear(x.to(torch.bfloat16), W.to(torch.bfloat16), bias=b, activation="silu", p=0.25, rng=RNG, y=y0, z=z)
        return float((g.double() * y0.double()).sum())

    loss(x, W, b)
    dx, dw, db = hkg.linear_backward(g, x.to(torch.bfloat16), W.to(torch.bfloat16), z=z, activation="silu", p=0.25, rng=RNG)
    # z is kept in bf16 (2^-8 of |z| <= 16, times silu'' <= 0.5), dz rounded to bf16
    gs = np.abs(f64(g)) / 0.75
    dz_off = gs * (2.0 ** -8 * np.abs(f64(z)) * 0.5 + 2.0 ** -8 * 1.1)
    noise = 2.0 ** -22 * float((g.abs() * y0.abs()).sum()) / h
    for i in range(0, N, 7):
        e = torch.zeros_like(b)
        e[i] = h
        d = (loss(x, W, b + e) - loss(x, W, b - e)) / (2 * h)
        assert abs(d - float(db[i])) <= dz_off[:, i].sum() + h * h / 6 * 0.15 * gs[:, i].sum() + noise
    for i, k in ((0, 0), (2, 5), (5, 15)):
        e = torch.zeros_like(x)
        e[i, k] = h
        d = (loss(x + e, W, b) - loss(x - e, W, b)) / (2 * h)
        w = np.abs(f64(W[:, k]))
        assert abs(d - float(dx[i, k])) <= dz_off[i] @ w + h * h / 6 * 0.15 * gs[i] @ w ** 3 + noise + 2.0 ** -8 * abs(d)
    for j, k in ((0, 0), (17, 5), (39, 15)):
        e = torch.zeros_like(W)
        e[j, k] = h
        d = (loss(x, W + e, b) - loss(x, W - e, b)) / (2 * h)
        a = np.abs(f64(x[:, k]))
        assert abs(d - float(dw[j, k])) <= dz_off[:, j] @ a + h * h / 6 * 0.15 * gs[:, j] @ a ** 3 + noise + 2.0 ** -8 * abs(d)


# ---- how they are called ----------------------------------------------------------------

def chain(x, W1, b1, W2, b2, r, rng, z):
    """A transformer's feed-forward block and its gradients, with every operator."""
    h = hkg.linear(x, W1, bias=b1, activation="gelu_tanh", z=z)
    y = hkg.linear(h, W2, bias=b2, residual=r, p=0.1, rng=rng)
    dh, dw2, db2 = hkg.linear_backward(y, h, W2, p=0.1, rng=rng)
    dx, dw1, db1 = hkg.linear_backward(dh, x, W1, z=z, activation="gelu_tanh")
    return (y, dx, dw1, db1, dw2, db2, hkg.dropout(y, 0.1, rng, residual=r))


def block(M=300, C=136, F=520, seed=1):
    return (normal(seed, M, C), normal(2, F, C, size=0.1), normal(3, F, kind="fp32"), normal(4, C, F, size=0.05), normal(5, C),
            normal(6, M, C))


def test_a_block_and_its_gradients():
    """The operators as a model uses them, against the same block in 64 bits: norms within
    2^-7, four roundings to bf16 of at most 2^-9 each in the mean."""
    x, W1, b1, W2, b2, r = block()
    z = torch.empty(300, 520, dtype=torch.bfloat16, device="cuda")
    got = chain(x, W1, b1, W2, b2, r, RNG, z)
    X, A1, B1, A2, B2, R = (f64(t) for t in (x, W1, b1, W2, b2, r))
    Z = X @ A1.T + B1
    H = ref.act(Z, "gelu_tanh")
    keep, s = ref.keep(300, 136, 0.1, RNG), ref.scale(0.1)
    Y = R + keep * s * (H @ A2.T + B2)
    D2 = keep * s * Y
    D1 = (D2 @ A2) * ref.slope(Z, "gelu_tanh")
    want = (Y, D1 @ A1, D1.T @ X, D1.sum(0), D2.T @ H, D2.sum(0), R + keep * s * Y)
    for i, (g, w) in enumerate(zip(got, want)):
        assert np.linalg.norm(f64(g) - w) <= 2.0 ** -7 * np.linalg.norm(w), i


def test_the_same_call_gives_the_same_bits():
    for args in (block(), block(2100, 2304, 72)):
        z = torch.empty(args[0].shape[0], args[1].shape[0], dtype=torch.bfloat16, device="cuda")
        a = chain(*args, RNG, z)
        for _ in range(3):
            for u, v in zip(a, chain(*args, RNG, z)):
                assert torch.equal(u, v)


@pytest.mark.parametrize("size", [(300, 136, 520), (2100, 2304, 72)])
def test_captured_and_replayed(size):
    """A graph of the block: replays, with eager work between them, take the inputs and the
    generator's numbers that are in its tensors then."""
    M, C, F = size
    args = list(block(M, C, F))
    rng = torch.tensor([3, 4], dtype=torch.int64, device="cuda")
    z = torch.empty(M, F, dtype=torch.bfloat16, device="cuda")
    chain(*args, rng, z)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        chain(*args, rng, z)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain(*args, rng, z)
    for i in range(4):
        args[0].copy_(normal(10 + i, M, C))
        rng.copy_(torch.tensor([i, 100 + i]))
        z2 = torch.empty_like(z)
        want = chain(*args, (i, 100 + i), z2)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for j, (u, v) in enumerate(zip(out, want)):
            assert torch.equal(u, v), (i, j)
        assert torch.equal(z, z2)


def test_on_another_stream():
    args = block()
    z = torch.empty(300, 520, dtype=torch.bfloat16, device="cuda")
    want = chain(*args, RNG, z)
    side = torch.cuda.Stream()
    x = args[0].clone()
    side.wait_stream(torch.cuda.current_stream())
    h = hkg.linear(x, args[1], bias=args[2], activation="gelu_tanh", z=z, stream=side)
    y = hkg.linear(h, args[3], bias=args[4], residual=args[5], p=0.1, rng=RNG, stream=side)
    g = hkg.linear_backward(y, h, args[3], p=0.1, rng=RNG, stream=side)
    o = hkg.dropout(y, 0.1, RNG, residual=args[5], stream=side)
    side.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(g[1], want[4]) and torch.equal(o, want[6])


def test_offsets_beyond_32_bits():
    """Rows so far apart that their offsets pass 2^31 elements and 2^32 bytes."""
    rows, pitch = 70001, 32768
    w = torch.empty(rows, pitch, dtype=torch.bfloat16, device="cuda")
    x = w[:, 100:140]
    x.copy_(normal(1, rows, 40))
    last = slice(rows - 50, rows)
    got = hkg.dropout(x, 0.5, RNG, out=x)
    want, tol = ref.dropout(f64(normal(1, rows, 40))[last], 0.5, RNG)
    keep = ref.keep(50, 40, 0.5, RNG, rows - 50)
    want = np.where(keep, f64(normal(1, rows, 40))[last] * 2.0, 0.0)
    close(got[last], want, 2.0 ** -8 * np.abs(want), "dropout")
    a, W, b = normal(2, rows, 16), normal(3, 40, 16), normal(4, 40)
    v = torch.empty(rows, pitch, dtype=torch.bfloat16, device="cuda")   # outputs may not share a span of bytes
    y, z = v[:, 201:241], w[:, 303:343]
    hkg.linear(a, W, bias=b, activation="silu", residual=y.copy_(x), p=0.5, rng=RNG, y=y, z=z)
    want, tol, zw, zt = ref.linear(f64(a[last]), f64(W), f64(b), "silu", f64(x[last]), 0.5, RNG, row0=rows - 50)
    close(y[last], want, tol, "y")
    close(z[last], zw, zt, "z")
    dy = y
    _, dw, db = hkg.linear_backward(dy, a, W, z=z, activation="silu", p=0.5, rng=RNG)
    _, dw2, db2 = hkg.linear_backward(dy.contiguous(), a, W, z=z.contiguous(), activation="silu", p=0.5, rng=RNG)
    assert torch.equal(dw, dw2) and torch.equal(db, db2)


def test_many_rows_and_columns():
    """More rows than one launch's grid has, and a single very long row."""
    x = normal(1, 600000, 8)
    got = hkg.dropout(x, 0.5, RNG)
    keep = ref.keep(40, 8, 0.5, RNG, 599960)
    np.testing.assert_array_equal(f64(got[-40:]), np.where(keep, 2 * f64(x[-40:]), 0.0))
    n = 5_000_001
    x = normal(2, 1, n)
    keep = ref.keep(1, n, 0.5, RNG)
    np.testing.assert_array_equal(f64(hkg.dropout(x, 0.5, RNG)), np.where(keep, 2 * f64(x), 0.0))
    W = normal(3, 2_000_003, 8)
    y = hkg.linear(normal(4, 1, 8), W, p=0.5, rng=RNG)
    keep = ref.keep(1, 2_000_003, 0.5, RNG)
    want, tol, _, _ = ref.linear(f64(normal(4, 1, 8)), f64(W))
    close(y, np.where(keep, 2 * want, 0.0), np.where(keep, 2 * tol, 0.0), "y")


def test_refused_calls_leave_their_outputs():
    x, W = normal(1, 8, 64), normal(2, 16, 64)
    y = torch.full((8, 16), 3.0, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(hkg.HkgError):
        hkg.linear(x[:, :60], W[:, :60].contiguous(), y=y)       # K is not a multiple of 8
    with pytest.raises(hkg.HkgError):
        hkg.linear(normal(1, 8, 72)[:, 4:68], W, y=y)            # rows of x are not 16-byte aligned
    with pytest.raises(hkg.HkgError):
        hkg.linear(x, W, y=x.view(-1)[:128].view(8, 16))         # y over x
    with pytest.raises(ValueError):
        hkg.linear(x, W, y=y, residual=torch.zeros(8, 16, device="cuda"))
    with pytest.raises(ValueError):
        hkg.linear(x, W, y=y, p=0.5)
    torch.cuda.synchronize()
    assert (y == 3.0).all()
