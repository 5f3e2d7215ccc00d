"""hkg_orthogonalize on gradients of many spectra against its iteration in 64 bits.

The tolerance is the output format's and knows nothing of how the operator
computes: bf16 rounds a value by up to 2^-8 of it, and the whole result may be off
by that, in the norm; an entry by that of itself and 2^-5 of the root mean square
entry (what a normally distributed error of 2^-8 of the norm reaches at eight
deviations)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("no GPU", allow_module_level=True)

import dense_gemm_fp8_amd as hkg  # noqa: E402

COEFFS, EPS = (3.4445, -4.7750, 2.0315), 1e-7


def gradient(kind, m, n, seed):
    """[m, n] in 64 bits, m <= n."""
    g = torch.Generator("cuda").manual_seed(seed)

    def randn(r, c):
        return torch.randn(r, c, dtype=torch.float64, device="cuda", generator=g)

    if kind.startswith("rank"):          # the gradient of a few tokens
        r = int(kind[4:])
        return randn(m, r) @ randn(r, n)
    if kind == "full":
        return randn(m, n)
    if kind == "one strong direction":
        x = randn(m, 1) @ randn(1, n)
        return x / x.norm() + 0.01 * randn(m, n) / (m * n) ** 0.5
    if kind == "constant":               # all entries near one value
        return 1 + 0.01 * randn(m, n)
    if kind == "few rows":               # experts, tokens or heads that took no part
        x = torch.zeros(m, n, dtype=torch.float64, device="cuda")
        x[::m // 8] = randn(len(x[::m // 8]), n)
        return x
    if kind == "unequal columns":
        return randn(m, n) * torch.exp(1.5 * randn(1, n))
    if kind == "unequal rows":           # six orders of magnitude
        return randn(m, n) * torch.logspace(0, -6, m, dtype=torch.float64, device="cuda")[:, None]
    if kind == "low rank and noise":
        return randn(m, 32) @ randn(32, n) + 1e-3 * randn(m, n)
    assert kind == "wide spectrum"       # singular values 1 .. 1e-4
    u, v = torch.linalg.qr(randn(m, m))[0], torch.linalg.qr(randn(n, m))[0]
    return (u * torch.logspace(0, -4, m, dtype=torch.float64, device="cuda")) @ v.t()


def iterated(G, steps=5, coeffs=COEFFS, eps=EPS):
    a, b, c = coeffs
    tall = G.shape[0] > G.shape[1]
    X = G.double().t() if tall else G.double()
    X = X / (X.norm() + eps)
    for _ in range(steps):
        A = X @ X.t()
        X = a * X + (b * A + c * (A @ A)) @ X
    return X.t() if tall else X


def check(got, want):
    off, size = (got.double() - want).abs(), want.norm()
    assert torch.isfinite(got).all()
    assert off.norm() <= 2.0 ** -8 * size, "%.5f of the norm off" % (off.norm() / size)
    rms = size / want.numel() ** 0.5
    worst = ((off - 2.0 ** -8 * want.abs()) / rms).max()
    assert worst <= 2.0 ** -5, "an entry is off by %.4f of the root mean square" % worst


KINDS = ["rank1", "rank4", "rank64", "full", "one strong direction", "constant", "few rows", "unequal columns",
         "unequal rows", "low rank and noise", "wide spectrum"]
# small blocks; 128-, 192- and 256-tiles; from 1.5 times as wide as high on; an update in two launches
SIZES = [(96, 200), (512, 2048), (768, 768), (700, 4500), (1500, 1600), (2304, 2600), (2048, 5632)]


@pytest.mark.parametrize("m,n", SIZES)
@pytest.mark.parametrize("kind", KINDS)
def test_spectra(kind, m, n):
    print("orth %s %dx%d" % (kind, m, n), flush=True)
    G = gradient(kind, m, n, m + n).float()
    check(hkg.orthogonalize(G), iterated(G))
    if m < 1000:                         # tall, and from bf16
        T = G.t().contiguous().to(torch.bfloat16)
        check(hkg.orthogonalize(T), iterated(T))


@pytest.mark.parametrize("kind", ["rank1", "rank4", "rank64", "one strong direction", "full"])
def test_a_large_matrix(kind):
    G = gradient(kind, 4096, 14336, 3).to(torch.bfloat16)
    check(hkg.orthogonalize(G), iterated(G))


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6, 7])
@pytest.mark.parametrize("m,n", [(256, 300), (640, 4500)])
def test_step_counts(m, n, steps):
    G = gradient("rank4", m, n, steps).float()
    check(hkg.orthogonalize(G, steps=steps), iterated(G, steps))


@pytest.mark.parametrize("m,n", [(130, 260), (640, 4500)])
def test_a_gradient_far_below_eps(m, n):
    # |G| / eps = 1e-6: the step is nearly linear, and entries of X are as small as 1e-9
    G = (1e-15 * gradient("full", m, n, 5) / (m * n) ** 0.5 * 100).float()
    check(hkg.orthogonalize(G), iterated(G))


@pytest.mark.parametrize("m,n", [(128, 384), (640, 4500)])
def test_singular_values_of_a_wide_spectrum(m, n):
    """Those of the result, taken along the input's singular vectors, within 2^-8 of
    the polynomial's (largest 1.2)."""
    g = torch.Generator("cuda").manual_seed(10)
    u = torch.linalg.qr(torch.randn(m, m, dtype=torch.float64, device="cuda", generator=g))[0]
    v = torch.linalg.qr(torch.randn(n, m, dtype=torch.float64, device="cuda", generator=g))[0]
    s = torch.logspace(0, -4, m, dtype=torch.float64, device="cuda")
    got = torch.diagonal(u.t() @ hkg.orthogonalize(((u * s) @ v.t()).float()).double() @ v)
    s = s / s.norm()
    for _ in range(5):
        s = COEFFS[0] * s + COEFFS[1] * s ** 3 + COEFFS[2] * s ** 5
    assert (got - s).abs().max() <= 2.0 ** -8
