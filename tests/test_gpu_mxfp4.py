"""GPU tests of the MXFP4 linear layer (include/hkg_ops.h) against the format's
definition in numpy and 64 bits (oracle/mxfp4.py): codes, scales and their
packed order bit for bit, products within the matrix instruction's summation
bound, and bit for bit where every sum is exact."""
import numpy as np
import pytest

from oracle import mxfp4 as ref
from oracle.parity import f32_to_bf16_rne

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("no GPU", allow_module_level=True)

import dense_gemm_fp8_amd as hkg  # noqa: E402

A, B = hkg.HKG_MX_OPERAND_A, hkg.HKG_MX_OPERAND_B


def say(msg):
    print(msg, flush=True)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def bits(t):
    return host(t.contiguous().view(torch.int16)).view(np.uint16)


def wild(seed, rows, K, dtype):
    """Values of every size: normal numbers times a power of two per block and
    row, exact rounding ties, zeros, subnormals, blocks of zeros."""
    g = np.random.Generator(np.random.PCG64(seed))
    x = g.standard_normal((rows, K))
    x *= np.exp2(g.integers(-20, 20, size=(rows, 1)))
    ties = g.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 4.0], size=x.shape) * np.sign(x)
    x = np.where(g.random(x.shape) < 0.2, ties, x)
    x = np.where(g.random(x.shape) < 0.1, 0.0, x)
    for b in range(0, K, 32):
        kind = g.random(rows)
        x[:, b:b + 32] = np.where((kind < 0.1)[:, None], 0.0, x[:, b:b + 32])
        tiny = np.exp2(g.integers(-150, -118, size=(rows, 1)).astype(np.float64))
        x[:, b:b + 32] = np.where(((kind > 0.1) & (kind < 0.2))[:, None], x[:, b:b + 32] * tiny, x[:, b:b + 32])
        huge = np.exp2(100.0)
        x[:, b:b + 32] = np.where((kind > 0.9)[:, None], np.clip(x[:, b:b + 32] * huge, -3e38, 3e38), x[:, b:b + 32])
    t = torch.from_numpy(x.astype(np.float32))
    return (t.to(torch.bfloat16) if dtype == "bf16" else t)


def check_form(codes, packed, want_codes, want_scales, operand, what):
    np.testing.assert_array_equal(host(codes), ref.pack_codes(want_codes), err_msg=what + " codes")
    want = ref.pack_scales(want_scales, operand)
    np.testing.assert_array_equal(host(packed)[:want.size], want, err_msg=what + " scales")


QUANT = [(1, 1), (1, 32), (3, 31), (2, 33), (17, 64), (128, 128), (129, 100), (130, 160), (31, 257), (300, 520)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,K", QUANT)
def test_quantize_bit_exact(rows, K, dtype):
    say("quantize %dx%d %s" % (rows, K, dtype))
    x = wild(100 + rows + K, rows, K, dtype)
    xs = x.float().numpy()
    c, s = ref.quantize(xs)
    ct, st = ref.quantize(xs.T)
    for op in (A, B):
        codes, packed = hkg.mxfp4_quantize(x.cuda(), op)
        check_form(codes, packed, c, s, op, "along K")
        codes, packed, codes_t, packed_t = hkg.mxfp4_quantize_both(x.cuda(), op, 1 - op)
        check_form(codes, packed, c, s, op, "both, along K")
        check_form(codes_t, packed_t, ct, st, 1 - op, "both, along rows")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_quantize_views_with_odd_strides_and_bases(dtype):
    big = wild(7, 140, 301, dtype).cuda()
    for r, k0, k1 in ((140, 0, 300), (77, 1, 200), (129, 3, 36), (5, 8, 8 + 256)):
        v = big[:r, k0:k1]
        say("quantize view %s" % (tuple(v.shape),))
        xs = v.float().cpu().numpy()
        codes, packed, codes_t, packed_t = hkg.mxfp4_quantize_both(v, A, B)
        check_form(codes, packed, *ref.quantize(xs), A, "view")
        check_form(codes_t, packed_t, *ref.quantize(xs.T), B, "view, transposed")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_nan_and_infinite_blocks(dtype):
    # only the block (along K, or along rows) that holds the bad value is NaN
    x = wild(9, 70, 130, dtype)
    x[0, 5], x[33, 64], x[69, 129] = float("nan"), float("inf"), float("-inf")
    xs = x.float().numpy()
    codes, packed, codes_t, packed_t = hkg.mxfp4_quantize_both(x.cuda(), A, B)
    check_form(codes, packed, *ref.quantize(xs), A, "nan")
    check_form(codes_t, packed_t, *ref.quantize(xs.T), B, "nan, transposed")
    v = host(hkg.mxfp4_dequantize(codes, packed, A, dtype=torch.float32))
    np.testing.assert_array_equal(v, ref.values(*ref.quantize(xs)))
    y = host(hkg.linear_mxfp4(x.cuda(), *one_weight(130)).float())
    rows = np.zeros(70, dtype=bool)
    rows[[0, 33, 69]] = True
    assert np.isnan(y[rows]).all() and np.isfinite(y[~rows]).all()


def one_weight(K):
    return hkg.mxfp4_quantize(torch.ones((5, K), dtype=torch.bfloat16, device="cuda"), B)


@pytest.mark.parametrize("rows,K", [(1, 32), (5, 96), (130, 160), (257, 1056)])
@pytest.mark.parametrize("operand", [A, B])
def test_dequantize_every_code_and_scale(rows, K, operand):
    g = np.random.Generator(np.random.PCG64(rows + K))
    codes = g.integers(0, 16, size=(rows, K), dtype=np.uint8)
    scales = g.integers(0, 256, size=(rows, K // 32), dtype=np.uint8)
    want = ref.values(codes, scales)
    with np.errstate(over="ignore"):
        want32 = want.astype(np.float32)         # 6 * 2^127 overflows in either type
    packed = hkg.mx_pack_scales(dev(scales), operand)
    got = host(hkg.mxfp4_dequantize(dev(ref.pack_codes(codes)), packed, operand, dtype=torch.float32))
    np.testing.assert_array_equal(got, want32)
    wide = torch.full((rows, K + 3), 7.0, dtype=torch.bfloat16, device="cuda")
    hkg.mxfp4_dequantize(dev(ref.pack_codes(codes)), packed, operand, out=wide[:, 1:K + 1])
    got = host(wide.float())
    np.testing.assert_array_equal(got[:, 1:K + 1], want32)
    assert (got[:, 0] == 7).all() and (got[:, K + 1:] == 7).all()


def mx_random(seed, rows, K, spread):
    """Codes of every value, scales 2^-spread .. 2^spread."""
    g = np.random.Generator(np.random.PCG64(seed))
    codes = g.integers(0, 16, size=(rows, ref.pad32(K)), dtype=np.uint8)
    codes[:, K:] = 0
    scales = g.integers(127 - spread, 128 + spread, size=(rows, ref.pad32(K) // 32)).astype(np.uint8)
    return codes, scales


def run_product(a, sa, b, sb):
    M, N = a.shape[0], b.shape[0]
    C = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    Cf = torch.full((M, N), float("nan"), dtype=torch.float32, device="cuda")
    hkg.gemm_mxfp4(dev(ref.pack_codes(a)), dev(ref.pack_codes(b)), hkg.mx_pack_scales(dev(sa), A),
                   hkg.mx_pack_scales(dev(sb), B), C, Cf)
    return bits(C), host(Cf)


def check_product(cb, cf, want, tol, what):
    bad = ~(np.abs(cf - want) <= tol)
    assert not bad.any(), "%s: %d of %d sums off, first at %s: %g for %g (tolerance %g)" % (
        what, bad.sum(), bad.size, np.argwhere(bad)[0], cf[bad][0], want[bad][0], tol[bad][0])
    np.testing.assert_array_equal(cb, f32_to_bf16_rne(cf), err_msg=what)


SHAPES = [(1, 1, 32), (1, 40, 64), (16, 32, 128), (17, 33, 160), (100, 300, 96), (128, 128, 256), (129, 257, 416),
          (256, 256, 512), (300, 520, 1056), (513, 260, 224), (640, 1100, 2048), (500, 1100, 352)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product_within_the_summation_bound(M, N, K):
    say("product %dx%dx%d" % (M, N, K))
    a, sa = mx_random(1 + M, M, K, 6)
    b, sb = mx_random(2 + N, N, K, 6)
    cb, cf = run_product(a, sa, b, sb)
    want, tol = ref.product(a, sa, b, sb)
    check_product(cb, cf, want, tol, "%dx%dx%d" % (M, N, K))


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product_exact_with_one_scale_per_row(M, N, K):
    # one scale for a row: every sum is a multiple of 1/4 of it, far below 2^24
    a, sa = mx_random(3 + M, M, K, 0)
    b, sb = mx_random(4 + N, N, K, 0)
    sa += (np.arange(M) % 5).astype(np.uint8)[:, None]
    sb -= (np.arange(N) % 7).astype(np.uint8)[:, None]
    cb, cf = run_product(a, sa, b, sb)
    want = ref.values(a, sa) @ ref.values(b, sb).T
    np.testing.assert_array_equal(cf, want)
    np.testing.assert_array_equal(cb, f32_to_bf16_rne(cf))


@pytest.mark.parametrize("M,N,K", [(4352, 4352, 96), (4300, 14300, 64), (1200, 6000, 288), (4096, 4096, 160)])
def test_product_of_many_tiles_exact(M, N, K):
    """256-tiles in one launch and split by rows or columns into two, edges
    included, every entry, against fp64 on the GPU (exact: one scale a row)."""
    a, sa = mx_random(13, M, K, 0)
    b, sb = mx_random(14, N, K, 0)
    sa += (np.arange(M) % 5).astype(np.uint8)[:, None]
    sb -= (np.arange(N) % 7).astype(np.uint8)[:, None]
    want = (dev(ref.values(a, sa)) @ dev(ref.values(b, sb)).t())
    args = (dev(ref.pack_codes(a)), dev(ref.pack_codes(b)), hkg.mx_pack_scales(dev(sa), A), hkg.mx_pack_scales(dev(sb), B))
    Cf = torch.full((M, N), float("nan"), dtype=torch.float32, device="cuda")
    C = hkg.gemm_mxfp4(*args, C_f32=Cf)
    assert torch.equal(Cf.double(), want)
    assert torch.equal(C, Cf.to(torch.bfloat16))
    assert torch.equal(hkg.gemm_mxfp4(*args), C)


def gpu_bound(va, vb, K):
    """|C_f32 - exact| from the summation bound, with a row's largest values in the
    place of a step's."""
    top = va.abs().amax(1)[:, None] * vb.abs().amax(1)[None, :]
    total = va.abs() @ vb.abs().t()
    return (K // 128 + 1) * (2.0 ** -6 * top + 2.0 ** -24 * total)


@pytest.mark.parametrize("M,N,K", [(1500, 1300, 544), (1100, 2777, 1184), (4352, 4352, 416), (4096, 8192, 288)])
def test_product_of_many_tiles_with_block_scales(M, N, K):
    """128- and 256-tiles with scales of their own in every block, every entry,
    against fp64 on the GPU."""
    a, sa = mx_random(15, M, K, 1)
    b, sb = mx_random(16, N, K, 1)
    va, vb = dev(ref.values(a, sa)), dev(ref.values(b, sb))
    Cf = torch.full((M, N), float("nan"), dtype=torch.float32, device="cuda")
    C = hkg.gemm_mxfp4(dev(ref.pack_codes(a)), dev(ref.pack_codes(b)), hkg.mx_pack_scales(dev(sa), A),
                       hkg.mx_pack_scales(dev(sb), B), C_f32=Cf)
    off = (Cf.double() - va @ vb.t()).abs()
    assert bool((off <= gpu_bound(va, vb, K)).all()), "largest error %g" % off.max()
    assert torch.equal(C, Cf.to(torch.bfloat16))


# few rows, 128-tiles and 256-tiles
@pytest.mark.parametrize("M,N", [(140, 150), (1500, 1300), (4200, 4000)])
def test_product_scale_nan_reaches_its_row_only(M, N):
    # also in the step that holds K's end, where the scales past it are read but not used
    for K in (96, 160, 256, 288):
        a, sa = mx_random(5, M, K, 2)
        b, sb = mx_random(6, N, K, 2)
        sa[7, -1] = sb[139, 0] = 255
        cb, cf = run_product(a, sa, b, sb)
        bad = np.zeros((M, N), dtype=bool)
        bad[7] = bad[:, 139] = True
        assert np.isnan(cf[bad]).all() and np.isfinite(cf[~bad]).all()


def test_product_writes_only_its_matrix():
    M, N, K = 130, 201, 128
    a, sa = mx_random(5, M, K, 0)
    b, sb = mx_random(6, N, K, 0)
    want = ref.values(a, sa) @ ref.values(b, sb).T
    pa, pb = hkg.mx_pack_scales(dev(sa), A), hkg.mx_pack_scales(dev(sb), B)
    for pitch in (201, 208, 211):
        big = torch.full((M + 2, pitch), 3.0, dtype=torch.bfloat16, device="cuda")
        hkg.gemm_mxfp4(dev(ref.pack_codes(a)), dev(ref.pack_codes(b)), pa, pb, C=big[:M, :N])
        got = host(big.float())
        np.testing.assert_array_equal(got[:M, :N], torch.from_numpy(want).to(torch.bfloat16).float().numpy())
        assert (got[M:] == 3).all() and (got[:, N:] == 3).all()


def test_empty_products():
    z = torch.zeros((0, 16), dtype=torch.uint8, device="cuda")
    one = torch.zeros((3, 16), dtype=torch.uint8, device="cuda")
    s = torch.full((512,), 127, dtype=torch.uint8, device="cuda")
    assert hkg.gemm_mxfp4(z, one, s, s).shape == (0, 3)
    assert hkg.gemm_mxfp4(one, z, s, s).shape == (3, 0)
    k0 = torch.zeros((3, 0), dtype=torch.uint8, device="cuda")
    assert (host(hkg.gemm_mxfp4(k0, k0, s, s).float()) == 0).all()
    x0 = torch.zeros((20, 0), dtype=torch.bfloat16, device="cuda")
    assert (host(hkg.linear_mxfp4(x0, k0, s).float()) == 0).all()


LINEAR = [(1, 1, 1), (1, 64, 33), (1, 1000, 4096), (2, 130, 100), (7, 257, 520), (16, 512, 1000), (17, 64, 96),
          (31, 300, 700), (100, 200, 257), (128, 384, 512), (257, 129, 640), (5, 8300, 160), (16, 8300, 97),
          (3, 70, 10272), (16, 40, 12000)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("M,N,K", LINEAR)
def test_linear(M, N, K, dtype):
    say("linear %dx%dx%d %s" % (M, N, K, dtype))
    g = np.random.Generator(np.random.PCG64(M + N + K))
    x = torch.from_numpy(g.standard_normal((M, K + 5)).astype(np.float32)).to(
        torch.bfloat16 if dtype == "bf16" else torch.float32)
    b, sb = mx_random(8 + N, N, K, 3)
    w, sw = dev(ref.pack_codes(b)), hkg.mx_pack_scales(dev(sb), B)
    for off in (0, 1):                              # off 1: unaligned rows
        v = x.cuda()[:, off:off + K]
        y = host(hkg.linear_mxfp4(v, w, sw).float())
        a, sa = ref.quantize(v.float().cpu().numpy())
        want, tol = ref.product(a, sa, b, sb)
        # the sum's own error, then half a bf16 step of the rounded result
        bad = ~(np.abs(y - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol))
        assert not bad.any(), "%d off" % bad.sum()


def test_linear_on_another_stream():
    K, N = 512, 300
    b, sb = mx_random(8, N, K, 3)
    w, sw = dev(ref.pack_codes(b)), hkg.mx_pack_scales(dev(sb), B)
    for M in (1, 40):
        x = torch.randn(M, K, device="cuda").to(torch.bfloat16)
        want = host(hkg.linear_mxfp4(x, w, sw).float())
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        ys = [hkg.linear_mxfp4(x, w, sw, stream=s) for _ in range(8)]
        torch.cuda.current_stream().wait_stream(s)
        for y in ys:
            np.testing.assert_array_equal(host(y.float()), want)


BACK = [(1, 1, 1), (32, 64, 32), (33, 70, 95), (100, 130, 257), (128, 256, 128), (300, 520, 200)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("M,N,K", BACK)
def test_backward_against_the_formula(M, N, K, dtype):
    say("backward %dx%dx%d %s" % (M, N, K, dtype))
    g = np.random.Generator(np.random.PCG64(M * N + K))
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    dy = torch.from_numpy(g.standard_normal((M, N)).astype(np.float32)).to(t).cuda()
    wt, swt = mx_random(11, K, N, 3)
    xt, sxt = mx_random(12, K, M, 3)
    args = (dev(ref.pack_codes(wt)), hkg.mx_pack_scales(dev(swt), B), dev(ref.pack_codes(xt)),
            hkg.mx_pack_scales(dev(sxt), B))
    dx, dw = hkg.linear_mxfp4_backward(dy, *args)
    d = dy.float().cpu().numpy()
    for got, (want, tol), what in ((dx, ref.product(*ref.quantize(d), wt, swt), "dx"),
                                   (dw, ref.product(*ref.quantize(d.T), xt, sxt), "dw")):
        got = host(got.float())
        bad = ~(np.abs(got - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol))
        assert not bad.any(), "%s: %d off" % (what, bad.sum())


@pytest.mark.parametrize("M,N,K", [(1100, 1300, 1500), (300, 2500, 2600), (4200, 4352, 4400)])
def test_backward_on_tiles(M, N, K):
    """Gradients whose products run as 128- or 256-tiles, in one launch or (few rows
    and tiles) in two, against fp64 on the GPU."""
    dy = torch.randn(M, N, device="cuda", generator=torch.Generator("cuda").manual_seed(M)).to(torch.bfloat16)
    q, s, qt, st = hkg.mxfp4_quantize_both(dy, A, A)          # checked bit for bit above
    W, x = torch.randn(N, K, device="cuda"), torch.randn(M, K, device="cuda")
    _, _, wt, swt = hkg.mxfp4_quantize_both(W, B, B)
    _, _, xt, sxt = hkg.mxfp4_quantize_both(x, A, B)
    dx, dw = hkg.linear_mxfp4_backward(dy, wt, swt, xt, sxt)
    v = lambda c, p, o: hkg.mxfp4_dequantize(c, p, o, dtype=torch.float32).double()  # noqa: E731
    for got, l, r, k in ((dx, v(q, s, A), v(wt, swt, B), N), (dw, v(qt, st, A), v(xt, sxt, B), M)):
        want = l @ r.t()
        tol = gpu_bound(l, r, k)
        assert bool(((got.double() - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol)).all())


def test_backward_against_differences():
    """L = sum(dy * y) with y = Q(x) W^T.  Inputs small integers with amax 4 in
    every block, so that Q(x) = x, W and dy are exact along every axis and so
    are the sums (whole numbers below 2^24); the loss is linear in each entry,
    so a central difference over a step that Q keeps (x +- 1 inside {-4..4}) is
    the gradient without error."""
    g = np.random.Generator(np.random.PCG64(3))
    M, N, K = 64, 96, 64

    def ints(r, c):
        v = g.integers(-2, 3, size=(r, c)).astype(np.float32)
        v[::32, :] = 4.0
        v[:, ::32] = 4.0
        return v

    x, W, dy = ints(M, K), ints(N, K), ints(M, N)
    t = lambda v: torch.from_numpy(v).to(torch.bfloat16).cuda()  # noqa: E731
    w, sw, wt, swt = hkg.mxfp4_quantize_both(t(W), B, B)
    _, _, xt, sxt = hkg.mxfp4_quantize_both(t(x), A, B)
    dx, dw = (host(v.float()) for v in hkg.linear_mxfp4_backward(t(dy), wt, swt, xt, sxt))

    def loss(xv, Wv):
        q, s = hkg.mxfp4_quantize(t(xv), A)
        qw, s2 = hkg.mxfp4_quantize(t(Wv), B)
        Cf = torch.empty((M, N), dtype=torch.float32, device="cuda")
        hkg.gemm_mxfp4(q, qw, s, s2, C_f32=Cf)
        return float((host(Cf).astype(np.float64) * dy).sum())

    for _ in range(12):
        m, n, k = g.integers(1, 32), g.integers(1, 32), g.integers(1, 32)   # not the 4s that set the scales
        for v, grad, at in ((x, dx, (m, k)), (W, dw, (n, k))):
            hi, lo = v.copy(), v.copy()
            hi[at] += 1
            lo[at] -= 1
            got = (loss(hi, W) - loss(lo, W)) / 2 if v is x else (loss(x, hi) - loss(x, lo)) / 2
            want = torch.tensor(got).to(torch.bfloat16).float().item()       # gradients come in bf16
            assert grad[at] == want


def test_graph_replays():
    """A captured quantise + product + few-token step gives the eager result on
    every replay, with other work between."""
    K, N, M = 512, 384, 200
    W = torch.randn(N, K, device="cuda").to(torch.bfloat16)
    x = torch.randn(M, K, device="cuda").to(torch.bfloat16)
    w, sw = hkg.mxfp4_quantize(W, B)

    def step():
        q, s = hkg.mxfp4_quantize(x, A)
        return hkg.gemm_mxfp4(q, w, s, sw), hkg.linear_mxfp4(x[:3], w, sw), hkg.linear_mxfp4(x, w, sw)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        x.copy_(torch.randn(M, K, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(out, step()):
            np.testing.assert_array_equal(bits(got), bits(want))


def test_offsets_past_32_bits():
    """40 000 000 rows of 64: elements of x, values and C lie past 2^31, bytes past 2^32, and
    the dequantising launch takes its rows in turns.  Row r is one pattern of exact
    values times 2^(r mod 7), so every result is known."""
    rows, K, N = 40_000_000, 64, 64
    g = np.random.Generator(np.random.PCG64(5))
    pattern = ref.MAGNITUDES[g.integers(0, 8, size=K)] * g.choice([-1.0, 1.0], size=K)
    pattern[[0, 40]] = 6.0                               # both blocks' scales: the row's power
    seven = pattern[None, :] * 2.0 ** np.arange(7)[:, None]
    some = torch.from_numpy(seven).to(torch.bfloat16).cuda()
    period = some.repeat(100_000, 1)                     # 700 000 rows, a multiple of 7
    x = torch.empty((rows, K), dtype=torch.bfloat16, device="cuda")

    def parts(t):
        for r in range(0, rows, len(period)):
            yield t[r:r + len(period)]

    for part in parts(x):
        part.copy_(period[:len(part)])
    codes, packed = hkg.mxfp4_quantize(x, A)
    v = hkg.mxfp4_dequantize(codes, packed, A)
    assert all(torch.equal(a, b) for a, b in zip(parts(v), parts(x)))
    del v, x
    w = ref.MAGNITUDES[g.integers(0, 8, size=(N, K))] * g.choice([-1.0, 1.0], size=(N, K))
    w[:, [0, 40]] = 6.0
    wc, ws = hkg.mxfp4_quantize(torch.from_numpy(w).float().cuda(), B)
    C = hkg.gemm_mxfp4(codes, wc, packed, ws)
    # sums of 64 products in steps of 1/4 below 64 * 36: exact in fp32, rounded once
    want = torch.from_numpy(seven @ w.T).float().to(torch.bfloat16).cuda().repeat(100_000, 1)
    assert all(torch.equal(part, want[:len(part)]) for part in parts(C))
